// Attention over the 4-bit key/value cache (layout: kv4.h) for many query rows of a sequence: prompts and
// chunks of them, bf16, on the fifth-generation tensor cores.
//
// The same formula as kv4_attn.h, arranged for a bound of arithmetic instead of bytes. An item is a (sequence, tile of
// 256 query rows, key/value head): a row is a (token, query head) pair, so the heads of a group share the keys and
// values of their tile. Its visible tokens are cut into stages of 128; all items' stages, end to end, are dealt out
// evenly and contiguously to one CTA per SM (an item counting kItemCost stages more), and an item that spans CTAs is
// joined by the CTA that arrives last, in CTA order.
//
// One CTA, 18 warps:
//   producer      bulk copies of the stage's packed units
//   8 converters  codes to 16-bit values o + s (n - 8) in the 128-byte-swizzled operand layout: K with a token per row,
//                 V^T with a channel per row (the packed value words hold two neighbouring tokens, which is the order
//                 that operand wants). Rounded once, to 11 bits, after a power of two has brought the largest key
//                 (value) so far below 2^14, so that no size of the keys and values is lost. Eight bits (bf16) would
//                 have needed no such factor, but cost the scores an error as large as the queries' own rounding.
//   MMA           one thread: S_x = Q_x K^T, O_x += P_x V for the two halves x of 128 rows
//   2 x 4 softmax a thread per row: running maximum (it moves only when passed by kSlack), weights
//                 p = 2^(y - m + 9) in 16 bits, written over S in tensor memory as the next product's operand
// While one half's softmax runs, the tensor core works on the other half. Tensor memory is full: S (128 columns) and O
// (hd columns) of both halves. A tile of at most 128 rows would leave one half idle: both then hold its queries, take
// alternate stages and are joined like the parts of an item.
//
// K's channels lie in the order 0 4 1 5 2 6 3 7 within every eight, as the codes unpack, and Q's with them; V^T's rows,
// the output's columns, in the order 0 2 .. 14 1 3 .. 15 within every sixteen, which the store undoes.
//
// Measured: 2 x 2048 tokens over 10007, 32 heads on 8, hd 128, gs 64: 459 us, 971 TFLOP/s (0.51 of a cuBLAS bf16
// product's rate). The converters set the pace: a stage takes them 1.8 to 1.9 us, with one softmax warp at work as with
// eight, half of it the dequantising, the rest the agreement on factors, waits and stores. A lane makes the scale and
// offset of one token ready for its warp (470 us; every lane for all tokens that it touches: 487 us). Eight requests of
// up to 20011 tokens with 30 rows a head: 87 us, of which 25 us do not depend on the lengths (start, queries, joining).
// What it cost to find: loops unrolled beyond the instruction cache took 1068 us, matrix instructions issued with
// operands in plain registers (110 cycles each instead of 45) 589 us; a thread fetching its own row of queries cost 6 us.
// Measured and dropped, against 482 us then: the row's scores all in registers (672 us), two threads per row (591 us),
// converters split into key and value warps (544 us), maximum and exponentials in one pass over the scores (523 us), bulk
// register moves between warpgroups and the next stage fetched into L2 ahead (no change); against 88 us for the 30 rows:
// the producer finding the factors from the scales ahead of the converters (97 us).
#include <cuda_fp16.h>

#include <atomic>

#include "kv4.h"
#include "pipe.h"
#include "tc.h"

namespace coli {

namespace {

constexpr int kTileTok = 128;                      // tokens of a stage
constexpr int kTileUnits = kTileTok / kKvUnit;     // 8
constexpr int kHalf = 128;                         // rows of a half (the instruction's M)
constexpr int kTileRows = 2 * kHalf;
constexpr int kConvWarps = kTileUnits;            // one unit each
constexpr int kSoftThreads = 2 * kHalf;
constexpr int kWarpConv = 8, kWarpMma = 16, kWarpLoad = 17;
constexpr int kTileThreads = 18 * 32;
constexpr int kSeqChunk = 512;                     // sequences whose stage counts are kept at a time
// Weights are 2^(y - m + kLift); the maximum m moves when a score passes it by kSlack (log2). 16 bits hold
// 2^(kLift + kSlack), and a move costs a pass over the output.
constexpr float kSlack = 6.f;
constexpr float kLift = 9.f, kUnlift = 1.f / 512.f;
constexpr float kInf = __builtin_huge_valf();
// What an item costs beside its stages, in stages: it counts in the shares, ahead of the item's first stage.
#ifndef COLI_KV4_TILE_COST
#define COLI_KV4_TILE_COST 6
#endif
constexpr int kItemCost = COLI_KV4_TILE_COST;

template <int HD, int NG>
struct Tile {
  static constexpr uint32_t kUnit = kv4_unit_bytes(HD, NG);
  static constexpr uint32_t kRaw = kTileUnits * kUnit;
  static constexpr uint32_t kQ = kHalf * HD * 2;     // one half's queries
  static constexpr uint32_t kK = kTileTok * HD * 2;  // keys, and values, of a stage
  static constexpr uint32_t kScales = kTileUnits * 2 * kKvUnit * NG * 4;  // a stage's scales and offsets in 16 bits
  static constexpr uint32_t kSmem = 1024 + 2 * kQ + 2 * kK + 2 * kK + kRaw + kScales;
  static constexpr int kWords = HD / 32, kWpg = kWords / NG;
};

struct TileArgs {
  Kv4View c;
  Kv4Plan p;
  const void* q;
  long long q_stride;
  int group;
  float scale;
  int window;
  void* out;
  long long out_stride;
  bool vec, vec_out;
  float* part;  // 2 per CTA: kTileRows x HD outputs, then kTileRows (maximum, sum) pairs
  int* count;
  int* err;
  uint64_t wait_ns;
  bool withhold;  // test hook: the call's first copy is withheld, and the waits on it give up
};

struct Item {
  int b, tile, head;
  int r0, m, len;
  int first, stages;  // first stage of kTileTok tokens, number of stages (at least 1)
  int lo;             // first token that a row of the tile sees
};

__device__ __forceinline__ int tiles_of(int m, int group) { return (int)(((long long)m * group + kTileRows - 1) / kTileRows); }

// Stages of tile k of a sequence: from the window of its first row to the position of its last.
__device__ __forceinline__ void tile_span(const TileArgs& a, int m, int len, int k, int& first, int& stages, int& lo) {
  const long long row0 = (long long)k * kTileRows;
  const long long all = (long long)m * a.group;
  const long long last_row = row0 + kTileRows - 1 < all - 1 ? row0 + kTileRows - 1 : all - 1;
  const int last = len - m + (int)(last_row / a.group);
  lo = kv4_from(len - m + (int)(row0 / a.group), a.window);
  first = last < 0 ? 0 : lo / kTileTok;
  stages = last < 0 ? 1 : last / kTileTok - first + 1;
}

__device__ __forceinline__ void load_seq(const TileArgs& a, Item& it) {
  int r1;
  kv4_rows(a.p, it.b, it.r0, r1, a.err);
  it.m = r1 - it.r0;
  it.len = kv4_len(a.p, a.c.page_log2, it.b, a.err);
}

// Stages (and item costs) of a whole sequence per head, by a warp.
__device__ __forceinline__ long long seq_stages(const TileArgs& a, int b) {
  Item it;
  it.b = b;
  load_seq(a, it);
  long long sum = 0;
  for (int k = threadIdx.x & 31, n = tiles_of(it.m, a.group); k < n; k += 32) {
    int first, stages, lo;
    tile_span(a, it.m, it.len, k, first, stages, lo);
    sum += stages + kItemCost;
  }
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// D[tmem] (+)= A[tmem] * B[smem]^T for one K step of 16, 16-bit A held two elements per column.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.u32 p, %4, 0; "
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}

// One lane of a converged warp, the same in every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ uint64_t uniform(uint64_t v) {
  return (uint64_t)__shfl_sync(0xffffffffu, (uint32_t)v, 0) | (uint64_t)__shfl_sync(0xffffffffu, (uint32_t)(v >> 32), 0) << 32;
}

// f16 A and B (K-major), f32 accumulator.
__host__ __device__ constexpr uint32_t f16_f32_idesc(uint32_t M, uint32_t N) {
  return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

#define COLI_R4(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3])
#define COLI_S4(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3])

// 32 consecutive 32-bit columns of this thread's lane; the load completes at tmem_wait_ld.
__device__ __forceinline__ void tmem_ld32(uint32_t at, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\ttcgen05.wait::ld.sync.aligned;"
      : COLI_R4(r, 0), COLI_R4(r, 4), COLI_R4(r, 8), COLI_R4(r, 12), COLI_R4(r, 16), COLI_R4(r, 20), COLI_R4(r, 24),
        COLI_R4(r, 28)
      : "r"(at)
      : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::COLI_S4(r, 0),
      COLI_S4(r, 4), COLI_S4(r, 8), COLI_S4(r, 12), COLI_S4(r, 16), COLI_S4(r, 20), COLI_S4(r, 24), COLI_S4(r, 28), "r"(at)
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::COLI_S4(r, 0),
      COLI_S4(r, 4), COLI_S4(r, 8), COLI_S4(r, 12), "r"(at)
      : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two binary32 values as one 64-bit register pair, and arithmetic on both at once.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  return (uint64_t)__float_as_uint(x) | (uint64_t)__float_as_uint(y) << 32;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& x, float& y) {
  x = __uint_as_float((uint32_t)v);
  y = __uint_as_float((uint32_t)(v >> 32));
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  return r;
}
__device__ __forceinline__ uint64_t add2_f32(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
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

__device__ __forceinline__ uint32_t bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ __half2 as_half2(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }

// The four code pairs of a word, (w >> 4 m) & 0x000f000f, as o + s (n - 8).
__device__ __forceinline__ void dequantise(uint32_t w, __half2 s, __half2 o, uint32_t (&v)[4]) {
  const __half2 bias = __floats2half2_rn(1032.f, 1032.f);
  const __half2 sixteenth = __floats2half2_rn(0.0625f, 0.0625f), bias16 = __floats2half2_rn(-72.f, -72.f);
  const uint32_t w8 = w >> 8;
  v[0] = bits(__hfma2(__hsub2(as_half2((w & 0x000f000fu) | 0x64006400u), bias), s, o));
  v[1] = bits(__hfma2(__hfma2(as_half2((w & 0x00f000f0u) | 0x64006400u), sixteenth, bias16), s, o));
  v[2] = bits(__hfma2(__hsub2(as_half2((w8 & 0x000f000fu) | 0x64006400u), bias), s, o));
  v[3] = bits(__hfma2(__hfma2(as_half2((w8 & 0x00f000f0u) | 0x64006400u), sixteenth, bias16), s, o));
}

template <int N>
__device__ __forceinline__ void lds_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 v = lds128(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = lds64(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    static_assert(N == 1, "1, 2 or 4 words");
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(smem_u32(p)) : "memory");
  }
}

__device__ __forceinline__ void sts128(uint32_t at, const uint32_t (&v)[4]) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}
__device__ __forceinline__ void sts32(uint32_t at, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

template <int N>
__device__ __forceinline__ void sts_words(uint32_t at, const uint32_t (&w)[N]) {
  if constexpr (N == 4)
    sts128(at, w);
  else if constexpr (N == 2)
    asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(at), "r"(w[0]), "r"(w[1]) : "memory");
  else
    sts32(at, w[0]);
}

// 2^(13 - floor(log2 x)), within what binary32 has: x times it lies in [2^13, 2^14).
__device__ __forceinline__ float below_2_14(float x) {
  const int ex = min(253, max(1, 127 + 13 + 127 - (int)(__float_as_uint(x) >> 23)));
  return __uint_as_float((uint32_t)ex << 23);
}

template <int HD, int NG>
__global__ void __launch_bounds__(kTileThreads, 1) kv4_tile_kernel(TileArgs a) {
  using T = Tile<HD, NG>;
  extern __shared__ uint8_t smem_raw[];
  // operand tiles on 1024-byte boundaries
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* s_q = smem;                    // [2 halves][HD / 64][128 rows][128 bytes]
  uint8_t* s_k = s_q + 2 * T::kQ;         // [2 stages][HD / 64][128 tokens][128 bytes]
  uint8_t* s_v = s_k + 2 * T::kK;         // [2 stages][2][HD channels][128 bytes = 64 tokens]
  uint8_t* s_raw = s_v + 2 * T::kK;       // [kTileUnits] packed units
  uint8_t* s_scale = s_raw + T::kRaw;     // [kTileUnits][keys, values][16 tokens][NG] scale | offset << 16
  __shared__ __align__(8) uint64_t raw_full, raw_empty, k_full[2], k_empty[2], v_full[2], v_empty[2], par_full[4],
      q_full[2], s_full[2], p_full[2], o_full[2];
  // per stage: 1 / key factor, value factor (0: none yet; below 0: s_nan names tokens of the stage), 1 / value factor
  __shared__ float s_par[4][3];
  __shared__ float s_big[2][kConvWarps];  // largest key and value of each unit, when a factor has to move
  __shared__ uint32_t s_nan[4][kConvWarps][NG];  // per stage, unit and group: tokens whose values are not finite
  __shared__ uint8_t s_nan_row[kSoftThreads];    // of a row's segment: groups of which it has seen such values
  __shared__ uint32_t s_tmem;
  __shared__ long long s_w[kSeqChunk];
  __shared__ long long s_at;
  __shared__ int s_start, s_start_tile, s_last;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < 2; i++) {
      mbar_init(&k_full[i], kConvWarps);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], kConvWarps);
      mbar_init(&v_empty[i], 1);
      mbar_init(&par_full[i], 1);
      mbar_init(&par_full[2 + i], 1);
      mbar_init(&q_full[i], 4);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_full[i], 1);
    }
    mbar_init(&raw_full, 1);
    mbar_init(&raw_empty, kConvWarps);
    mbar_fence_init();
  }
  griddep_launch_dependents();
  griddep_wait();

  // ---- deal the stages out ----
  const int heads = a.c.heads;
  long long total = 0;
  for (int base = 0; base < a.p.B; base += kSeqChunk) {
    const int n = min(kSeqChunk, a.p.B - base);
    for (int i = warp; i < n; i += kTileThreads / 32) {
      const long long s = seq_stages(a, base + i) * heads;
      if (lane == 0) s_w[i] = s;
    }
    __syncthreads();
    long long sum = 0;
    for (int i = lane; i < n; i += 32) sum += s_w[i];
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    total += sum;
    if (base + kSeqChunk < a.p.B) __syncthreads();
  }
  const long long per = (total + gridDim.x - 1) / gridDim.x;
  const long long w0 = per * blockIdx.x, w1 = w0 + per < total ? w0 + per : total;
  if (w0 >= w1) return;  // uniform in the CTA: nothing allocated, nothing in flight
  {
    long long before = 0;
    bool found = false;
    for (int base = 0; base < a.p.B && !found; base += kSeqChunk) {
      const int n = min(kSeqChunk, a.p.B - base);
      if (a.p.B > kSeqChunk) {  // otherwise s_w still holds them
        __syncthreads();
        for (int i = warp; i < n; i += kTileThreads / 32) {
          const long long s = seq_stages(a, base + i) * heads;
          if (lane == 0) s_w[i] = s;
        }
        __syncthreads();
      }
      for (int i0 = 0; i0 < n && !found; i0 += 32) {
        const long long mine = i0 + lane < n ? s_w[i0 + lane] : 0;
        long long inc = mine;
        for (int o = 1; o < 32; o <<= 1) {
          const long long v = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += v;
        }
        const bool here = mine > 0 && before + inc - mine <= w0 && w0 < before + inc;
        const unsigned who = __ballot_sync(0xffffffffu, here);
        if (who) {
          found = true;
          if (here && warp == 0) {
            s_start = base + i0 + lane;
            s_at = before + inc - mine;
          }
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
      }
    }
  }
  __syncthreads();
  Item it;
  it.b = s_start;
  load_seq(a, it);
  if (warp == 0) {  // the tile of the sequence in which the share starts
    long long at = s_at;
    const int n = tiles_of(it.m, a.group);
    for (int k0 = 0; k0 < n; k0 += 32) {
      int first, stages = 0, lo;
      if (k0 + lane < n) tile_span(a, it.m, it.len, k0 + lane, first, stages, lo);
      const long long mine = k0 + lane < n ? (long long)(stages + kItemCost) * heads : 0;
      long long inc = mine;
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      const bool here = mine > 0 && at + inc - mine <= w0 && w0 < at + inc;
      if (here) {
        s_start_tile = k0 + lane;
        s_at = at + inc - mine;
      }
      if (__any_sync(0xffffffffu, here)) break;
      at += __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  if (warp == kWarpMma) tmem_alloc(&s_tmem, 512);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = s_tmem;

  it.tile = s_start_tile;
  tile_span(a, it.m, it.len, it.tile, it.first, it.stages, it.lo);
  const long long local = w0 - s_at;
  it.head = (int)(local / (it.stages + kItemCost));
  // below 0: in the item's cost. w counts stages and costs.
  int stage = (int)(local % (it.stages + kItemCost)) - kItemCost;
  long long w = w0;
  auto more = [&]() {  // past the item's cost; false at the end of the share
    if (stage < 0) w -= stage, stage = 0;
    return w < w1;
  };
  auto next_item = [&]() {  // w < w1 guarantees that there is one
    if (++it.head < heads) return;
    it.head = 0;
    if (++it.tile >= tiles_of(it.m, a.group)) {
      it.tile = 0;
      do {
        it.b++;
        load_seq(a, it);
      } while (it.m == 0 && it.b + 1 < a.p.B);
    }
    tile_span(a, it.m, it.len, it.tile, it.first, it.stages, it.lo);
  };
  auto rows_here = [&]() { return (int)min((long long)kTileRows, (long long)it.m * a.group - (long long)it.tile * kTileRows); };
  bool alive = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (alive && !mbar_wait_suspend(bar, parity, a.wait_ns)) {
      set_error(a.err, COLI_E_TIMEOUT);
      alive = false;  // void from here on, but nothing hangs
    }
  };

  if (warp == kWarpLoad) {
    // ------------------------------------ producer ------------------------------------
    const int page_tok = 1 << a.c.page_log2;
    int cached_b = -1, cached_from = 0, pages = 0;
    uint32_t fills = 0;
    for (uint32_t n = 0; more(); n++) {
      const int tok = (it.first + stage) * kTileTok;
      const int units = min(kTileUnits, max(0, (it.len - tok + kKvUnit - 1) / kKvUnit));
      const int page = tok >> a.c.page_log2;
      const int per_copy = min(kTileUnits, page_tok / kKvUnit);  // units
      const int copies = (units + per_copy - 1) / per_copy;      // at most 8
      if (copies > 0 && (it.b != cached_b || page < cached_from || page + copies > cached_from + 32)) {
        cached_b = it.b;
        cached_from = page;
        pages = page + lane < a.p.table_stride ? __ldcg(a.p.table + (size_t)it.b * a.p.table_stride + page + lane) : 0;
      }
      wait(&raw_empty, (n & 1) ^ 1);
      if (__any_sync(0xffffffffu, !alive)) break;
      const bool held = a.withhold && w == kItemCost;
      if (lane == 0 && !held) mbar_arrive_expect_tx(&raw_full, units * T::kUnit);
      fills += !held;
      __syncwarp();
      int pg = __shfl_sync(0xffffffffu, pages, (page - cached_from + lane) & 31);
      if (lane < copies && !held) {
        if (pg < 0 || pg >= a.c.pages) {
          if (tok + (lane + 1) * per_copy * kKvUnit > it.lo) set_error(a.err, COLI_E_RANGE);
          pg = 0;  // some page of the cache in its place; no row sees a page that its window has left
        }
        const int take = min(per_copy, units - lane * per_copy);
        const uint8_t* src = a.c.base + (((size_t)pg * heads + it.head) * (size_t)(page_tok / kKvUnit) +
                                         (tok & (page_tok - 1)) / kKvUnit) * T::kUnit;
        bulk_g2s(s_raw + lane * per_copy * T::kUnit, src, take * T::kUnit, &raw_full);
      }
      w++;
      if (++stage == it.stages) {
        stage = -kItemCost;
        if (w < w1) next_item();
      }
    }
    if (fills > 0) mbar_wait(&raw_full, (fills - 1) & 1);  // no copy is in flight when the CTA ends
  } else if (warp == kWarpMma) {
    // -------------------------------------- MMA --------------------------------------
    // One elected lane issues. Its operands are the same in the whole warp, and made so visibly (shuffles): they
    // then live in uniform registers, where the instruction wants them.
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t dq0 = uniform(sw128_kmajor_desc(s_q)), dk = uniform(sw128_kmajor_desc(s_k)), dv0 = uniform(sw128_kmajor_desc(s_v));
    if (elect_one()) {
      constexpr uint32_t kIdS = f16_f32_idesc(kHalf, kTileTok), kIdO = f16_f32_idesc(kHalf, HD);
      uint32_t n = 0, ns[2] = {0, 0}, nseg[2] = {0, 0};  // stages, stages and segments of each half
      auto scores = [&](int x, uint32_t stage_n) {
#pragma unroll
        for (int k = 0; k < HD / 16; k++) {
          // a descriptor's address field counts 16 bytes
          const uint64_t da = dq0 + (uint32_t)(x * (T::kQ >> 4)) + (k / 4) * (kHalf * 8) + (k % 4) * 2;
          tc_mma_bf16(tm + x * kTileTok, da, dk + (stage_n & 1) * (T::kK >> 4) + (k / 4) * (kTileTok * 8) + (k % 4) * 2, kIdS, k != 0);
        }
        tc_commit(&s_full[x]);
      };
      auto output = [&](int x, uint32_t stage_n, bool fresh) {
        const uint64_t dv = dv0 + (stage_n & 1) * (T::kK >> 4);
#pragma unroll
        for (int k = 0; k < kTileTok / 16; k++)
          mma_ts(tm + 2 * kTileTok + x * HD, tm + x * kTileTok + k * 8, dv + (k / 4) * (HD * 8) + (k % 4) * 2, kIdO,
                 !(fresh && k == 0));
      };
      while (more()) {
        const int n_here = (int)min((long long)(it.stages - stage), w1 - w);
        const bool split = rows_here() <= kHalf;
        const int halves = split && n_here == 1 ? 1 : 2;  // with work here
        for (int x = 0; x < halves; x++) {
          wait(&q_full[x], nseg[x] & 1);
          nseg[x]++;
        }
        if (split) {
#pragma unroll 1
          for (int x = 0; x < halves; x++) {
            wait(&k_full[(n + x) & 1], ((n + x) >> 1) & 1);
            tc_fence_after_sync();
            scores(x, n + x);
            tc_commit(&k_empty[(n + x) & 1]);
          }
#pragma unroll 1
          for (int j = 0; j < n_here; j++, n++) {
            const int x = j & 1;
            wait(&v_full[n & 1], (n >> 1) & 1);
            wait(&p_full[x], ns[x] & 1);
            ns[x]++;
            tc_fence_after_sync();
            output(x, n, j < 2);
            tc_commit(&v_empty[n & 1]);
            if (j + 2 < n_here) {
              wait(&k_full[n & 1], ((n + 2) >> 1) & 1);
              tc_fence_after_sync();
              scores(x, n + 2);
              tc_commit(&k_empty[n & 1]);
            } else {
              tc_commit(&o_full[x]);
            }
          }
        } else {
          wait(&k_full[n & 1], (n >> 1) & 1);
          tc_fence_after_sync();
#pragma unroll 1
          for (int x = 0; x < 2; x++) scores(x, n);
          tc_commit(&k_empty[n & 1]);
#pragma unroll 1
          for (int j = 0; j < n_here; j++, n++) {
            wait(&v_full[n & 1], (n >> 1) & 1);
#pragma unroll 1
            for (int x = 0; x < 2; x++) {
              wait(&p_full[x], ns[x] & 1);
              ns[x]++;
              tc_fence_after_sync();
              output(x, n, j == 0);
              if (j + 1 == n_here) tc_commit(&o_full[x]);
              if (x == 1) tc_commit(&v_empty[n & 1]);
              if (j + 1 < n_here) {  // the next stage's scores go over the weights that the product above reads first
                if (x == 0) {
                  wait(&k_full[(n + 1) & 1], ((n + 1) >> 1) & 1);
                  tc_fence_after_sync();
                }
                scores(x, n + 1);
                if (x == 1) tc_commit(&k_empty[(n + 1) & 1]);
              }
            }
          }
        }
        w += n_here;
        stage += n_here;
        if (stage == it.stages) {
          stage = -kItemCost;
          if (w < w1) next_item();
        }
      }
      // the last arrivals on these barriers come before the CTA's memory goes, whatever has been given up
      mbar_wait(&k_empty[(n - 1) & 1], ((n - 1) >> 1) & 1);
      mbar_wait(&v_empty[(n - 1) & 1], ((n - 1) >> 1) & 1);
    }
    __syncwarp();
  } else if (warp >= kWarpConv) {
    // ----------------------------------- converters -----------------------------------
    // A warp converts one unit, which it first takes into registers, so that the next copy can start.
    const int cw = warp - kWarpConv, r = lane >> 2, cc = lane & 3;
    const uint32_t k_base0 = smem_u32(s_k) + (cw * 16 + r) * 128;
    const uint32_t v_base0 = smem_u32(s_v) + (cw / 4) * (HD * 128) + r * 128 + cc * 4;
    const uint8_t* unit = s_raw + cw * T::kUnit;
    const uint8_t* scales_at = s_scale + cw * (2 * kKvUnit * NG * 4);
    const uint32_t scales = smem_u32(scales_at);
    float kmul = 0.f, vmul = 0.f;  // keys and values are multiplied by them; they only shrink within a segment
    float kinv = 1.f, vinv = 0.f;  // 1 / kmul, 1 / vmul
    for (uint32_t n = 0; more(); n++) {
      if (n == 0 || stage == 0) kmul = vmul = vinv = 0.f, kinv = 1.f;
      const int left = it.len - (it.first + stage) * kTileTok - cw * 16;  // tokens of this unit that exist
      wait(&raw_full, n & 1);
      // codes of tokens r, r + 8 (keys) and of token pairs c, c + 4 (values); scales and offsets of one token, keys' in
      // lanes 0..15, values' in lanes 16..31: made ready once, and shared through s_scale
      uint32_t kw[2][T::kWords], vw[2][T::kWords], sc[NG];
#pragma unroll
      for (int h = 0; h < 2; h++) {
        lds_words(unit + h * 32 * T::kWords * 4 + lane * T::kWords * 4, kw[h]);
        lds_words(unit + kv4_v_at(HD, NG) + h * 4 * HD + lane * T::kWords * 4, vw[h]);
      }
      lds_words(unit + (lane < 16 ? kv4_kscale_at(HD) : kv4_vscale_at(HD, NG)) + (lane & 15) * NG * 4, sc);
      __syncwarp();
      if (lane == 0) mbar_arrive(&raw_empty);
      // tokens that no row of the tile sees hold anything
      const int before = max(0, it.lo - (it.first + stage) * kTileTok - cw * 16);
      const bool live = (uint32_t)((lane & 15) - before) < (uint32_t)max(0, left - before);
      float big = 0.f;  // the largest |o| + 8 s of the token; not a number, or infinite, if a key or value is not finite
#pragma unroll
      for (int g = 0; g < NG; g++) big = max_nan(big, fmaf(8.f, lo_bf16(sc[g]), fabsf(hi_bf16(sc[g]))));
      if (!live) big = 0.f;
      auto too_big = [](float x, float mul) { return mul == 0.f ? !(x <= 0.f) : !(x * mul < 16384.f); };
      if (named_sync_or(2, kConvWarps * 32, too_big(big, lane < 16 ? kmul : vmul))) {
        // What is not finite stays out of the factors. A key becomes NaN, as its scores then do; a value becomes 0, and is
        // noted for the rows that see it.
        uint32_t broken = 0;
        big = 0.f;
#pragma unroll
        for (int g = 0; g < NG; g++) {
          if (kv4_broken(sc[g])) {
            broken |= live && lane >= 16 ? 1u << g : 0u;
            sc[g] = lane < 16 ? 0x7fc00000u : 0u;
          } else if (live) {
            big = fmaxf(big, fmaf(8.f, lo_bf16(sc[g]), fabsf(hi_bf16(sc[g]))));
          }
        }
        float kbig = __uint_as_float(__reduce_max_sync(0xffffffffu, lane < 16 ? __float_as_uint(big) : 0u));
        float vbig = __uint_as_float(__reduce_max_sync(0xffffffffu, lane < 16 ? 0u : __float_as_uint(big)));
        if (lane == 0) {
          s_big[0][cw] = kbig;
          s_big[1][cw] = vbig;
        }
        const bool noted = named_sync_or(2, kConvWarps * 32, broken != 0);  // the same in all converters
#pragma unroll
        for (int i = 0; i < kConvWarps; i++) {
          kbig = fmaxf(kbig, s_big[0][i]);
          vbig = fmaxf(vbig, s_big[1][i]);
        }
        if (noted) {
          wait(&k_empty[n & 1], ((n >> 1) & 1) ^ 1);  // the softmax of four stages ago is long done
#pragma unroll
          for (int g = 0; g < NG; g++) {
            const unsigned tokens = __ballot_sync(0xffffffffu, broken >> g & 1) >> 16;
            if (lane == 0) s_nan[n & 3][cw][g] = tokens;
          }
          named_sync(2, kConvWarps * 32);
        }
        if (too_big(kbig, kmul)) kmul = below_2_14(kbig), kinv = 1.f / kmul;
        if (too_big(vbig, vmul)) vmul = below_2_14(vbig), vinv = 1.f / vmul;
        if (noted) {
          if (vmul == 0.f) vmul = __uint_as_float(253u << 23), vinv = 1.f / vmul;
          vinv = -vinv;  // until it is passed on
        }
      }
      {
        const float mul = lane < 16 ? kmul : vmul;
#pragma unroll
        for (int g = 0; g < NG; g++) {
          const uint32_t ready = bits(__floats2half2_rn(lo_bf16(sc[g]) * mul, hi_bf16(sc[g]) * mul));
          sc[g] = live && (lane < 16 || vmul != 0.f) ? ready : 0u;
        }
        sts_words(scales + lane * NG * 4, sc);
        __syncwarp();
      }
      // ---- keys: odd tokens store the words of a pair in the other order: eight lanes then cover all banks ----
      wait(&k_empty[n & 1], ((n >> 1) & 1) ^ 1);
      if (cw == 0 && lane == 0) {  // the softmax of four stages ago is long done
        s_par[n & 3][0] = kinv;
        s_par[n & 3][1] = copysignf(vmul, vinv);
        s_par[n & 3][2] = fabsf(vinv);
        mbar_arrive(&par_full[n & 3]);
      }
      vinv = fabsf(vinv);
      const uint32_t k_base = k_base0 + (n & 1) * T::kK;
      const int odd = r & 1;
#pragma unroll
      for (int h = 0; h < 2; h++) {
        __half2 s[NG], o[NG];
        lds_words(scales_at + (r + 8 * h) * NG * 4, sc);
#pragma unroll
        for (int g = 0; g < NG; g++) s[g] = as_half2(__byte_perm(sc[g], 0, 0x1010)), o[g] = as_half2(__byte_perm(sc[g], 0, 0x3232));
#pragma unroll
        for (int i = 0; i < T::kWords; i++) {
          const int j = i ^ 1;
          uint32_t v[4];
          dequantise(odd ? kw[h][j] : kw[h][i], odd ? s[j / T::kWpg] : s[i / T::kWpg], odd ? o[j / T::kWpg] : o[i / T::kWpg], v);
          sts128(k_base + h * 8 * 128 + (i / 2) * (kTileTok * 128) + (((((i & 1) ^ odd) * 4 + cc) ^ r) << 4), v);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&k_full[n & 1]);
      // ---- values ----
      wait(&v_empty[n & 1], ((n >> 1) & 1) ^ 1);
      const uint32_t v_base = v_base0 + (n & 1) * T::kK;
#pragma unroll
      for (int h = 0; h < 2; h++) {
        __half2 s[NG], o[NG];
        uint32_t sc1[NG];
        lds_words(scales_at + (16 + 2 * cc + 8 * h) * NG * 4, sc);
        lds_words(scales_at + (16 + 2 * cc + 8 * h + 1) * NG * 4, sc1);
#pragma unroll
        for (int g = 0; g < NG; g++)
          s[g] = as_half2(__byte_perm(sc[g], sc1[g], 0x5410)), o[g] = as_half2(__byte_perm(sc[g], sc1[g], 0x7632));
        const uint32_t at = v_base + ((((cw % 4) * 2 + h) ^ r) << 4);  // the chunk of eight tokens
#pragma unroll
        for (int i = 0; i < T::kWords; i++) {
          uint32_t v[4];
          dequantise(vw[h][i], s[i / T::kWpg], o[i / T::kWpg], v);
#pragma unroll
          for (int j = 0; j < 4; j++) sts32(at + ((2 * i + (j >> 1)) * 16 + (j & 1) * 8) * 128, v[j]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&v_full[n & 1]);
      w++;
      if (++stage == it.stages) {
        stage = -kItemCost;
        if (w < w1) next_item();
      }
    }
  } else {
    // ------------------------------------- softmax -------------------------------------
    const int x = warp >> 2;                 // half
    const int row = tid & (kTileRows - 1);   // of the tile
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lanes + x * kTileTok, t_o = tmem + lanes + 2 * kTileTok + x * HD;
    uint32_t n = 0, ns = 0, nseg = 0;
    float fac0 = 0.f;
    // This row's queries of the item at the cursor, into shared memory: a power of two brings the largest to
    // [2^14, 2^15), and fac0 takes the scores back, in log2 units.
    auto load_queries = [&]() {
      const int row_n = rows_here(), n_here = (int)min((long long)(it.stages - stage), w1 - w);
      const bool split = row_n <= kHalf;
      if (split && x == 1 && n_here == 1) return;
      const int lrow = split ? row & (kHalf - 1) : row;
      if ((lrow & ~31) >= row_n) {  // a warp without rows: whatever its queries hold, nothing reads their results
        if (lane == 0) mbar_arrive(&q_full[x]);
        return;
      }
      // Lanes lie along a row, HD / 8 of them: a thread fetching its own row would touch 32 lines with every load.
      constexpr int kAcross = HD / 8, kAtOnce = 32 / kAcross;  // lanes of a row, rows of a load
      const long long q_row = (long long)it.tile * kTileRows + min(lrow, row_n - 1);
      const long long mine = (it.r0 + q_row / a.group) * a.q_stride + (it.head * a.group + q_row % a.group) * HD;
      const int ch = lane % kAcross, sub = lane / kAcross;
      uint4 v[kAcross];  // all in flight
#pragma unroll
      for (int i = 0; i < kAcross; i++) {
        const unsigned short* src = static_cast<const unsigned short*>(a.q) + __shfl_sync(0xffffffffu, mine, i * kAtOnce + sub) + 8 * ch;
        if (a.vec) {
          v[i] = __ldcg(reinterpret_cast<const uint4*>(src));
        } else {
          uint32_t e[4];
#pragma unroll
          for (int j = 0; j < 4; j++) e[j] = __ldcg(src + 2 * j) | ((uint32_t)__ldcg(src + 2 * j + 1) << 16);
          v[i] = make_uint4(e[0], e[1], e[2], e[3]);
        }
      }
      const uint32_t dst = smem_u32(s_q) + x * T::kQ + (ch / 8) * (kHalf * 128);
      const int first_row = row & (kHalf - 1) & ~31;
      float inv = 1.f;  // of this thread's row
      bool broken = false;
#pragma unroll
      for (int i = 0; i < kAcross; i++) {
        const uint32_t qw[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        uint32_t amax = 0;
#pragma unroll
        for (int j = 0; j < 4; j++) amax = max(amax, max(qw[j] & 0x7fffu, qw[j] >> 16 & 0x7fffu));
#pragma unroll
        for (int o = 1; o < kAcross; o <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const int ex = min(253, max(1, 127 + 14 + 127 - (int)(amax >> 7)));
        float mult = amax == 0 ? 1.f : __uint_as_float((uint32_t)ex << 23);
        const float of = __shfl_sync(0xffffffffu, amax == 0 ? 1.f : __uint_as_float((uint32_t)(254 - ex) << 23), lane % kAtOnce * kAcross);
        if (lane / kAtOnce == i) inv = of;
        if (a.scale < 0.f) mult = -mult;
        if (amax >= 0x7f80u) mult = __uint_as_float(0x7fc00000u);
        broken = broken || amax >= 0x7f80u;  // rows past the end repeat the last
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; j++) f[2 * j] = lo_bf16(qw[j]) * mult, f[2 * j + 1] = hi_bf16(qw[j]) * mult;
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; j++) o[j] = bits(__floats2half2_rn(f[j], f[j + 4]));
        const int at = first_row + i * kAtOnce + sub;
        sts128(dst + at * 128 + (((ch % 8) ^ (at & 7)) << 4), o);
      }
      if (broken) set_error(a.err, COLI_E_NONFINITE);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[x]);
      fac0 = fabsf(a.scale) * 1.4426950408889634f * inv;
    };
    if (more()) load_queries();
    while (more()) {
      const Item at = it;  // the item of this segment; the cursor moves on before its results are stored
      const long long item_at = w - stage;  // where the item's first stage is in what was dealt out
      const int n_here = (int)min((long long)(it.stages - stage), w1 - w);
      const int row_n = rows_here();
      // A tile of at most 128 rows: both halves hold its queries and take alternate stages.
      const bool split = row_n <= kHalf;
      const bool active = !split || x == 0 || n_here > 1;
      const int lrow = split ? row & (kHalf - 1) : row;
      const long long q_row = (long long)at.tile * kTileRows + min(lrow, row_n - 1);  // rows past the end repeat the last
      const int pos = at.len - at.m + (int)(q_row / a.group);
      const bool rows = (lrow & ~31) < row_n;  // a warp without rows only keeps the products' pace
      float mf = -kInf, l = 0.f, vmul = 0.f, unscale = 0.f;
      s_nan_row[tid] = 0;
      if (active && !rows) {
        for (int j = split ? x : 0; j < n_here; j += split ? 2 : 1, ns++) {
          wait(&s_full[x], ns & 1);
          if (lane == 0) mbar_arrive(&p_full[x]);
        }
      } else if (active) {
        const int step = split ? 2 : 1, j0 = split ? x : 0;
        for (int j = j0; j < n_here; j += step, ns++) {
          const int t0 = (at.first + stage + j) * kTileTok;
          wait(&s_full[x], ns & 1);
          tc_fence_after_sync();
          // The scores are there, so their stage's factors are: this wait does not wait, and comes second because a
          // half that has skipped stages could take an earlier phase of the barrier for this one.
          const uint32_t par = (n + j) & 3;
          wait(&par_full[par], ((n + j) >> 2) & 1);
          // kept above 0, so that struck-out scores (minus infinity) stay so
          const float fac = fmaxf(fac0 * s_par[par][0], 1e-37f);
          float vnow = s_par[par][1];
          unscale = s_par[par][2];
          // columns [c0, c1) are visible to this row; the others are struck out where they lie
          const int c1 = min(kTileTok, max(0, pos - t0 + 1));
          const int c0 = min(kTileTok, max(0, kv4_from(pos, a.window) - t0));
          uint32_t sv[32];
          if (__any_sync(0xffffffffu, c1 < kTileTok || c0 > 0)) {
#pragma unroll 1
            for (int k = 0; k < kTileTok; k += 32) {
              tmem_ld32(t_s + k, sv);
#pragma unroll
              for (int i = 0; i < 32; i++)
                if (k + i < c0 || k + i >= c1) sv[i] = 0xff800000u;
              tmem_st32(t_s + k, sv);
            }
            tmem_wait_st();
          }
          float mx = -kInf;
#pragma unroll 1
          for (int k = 0; k < kTileTok; k += 32) {
            tmem_ld32(t_s + k, sv);
            float m4[4] = {mx, -kInf, -kInf, -kInf};
#pragma unroll
            for (int i = 0; i < 32; i += 2)
              m4[i >> 1 & 3] = max3(m4[i >> 1 & 3], __uint_as_float(sv[i]), __uint_as_float(sv[i + 1]));
            mx = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]);
          }
          const float top = mx == -kInf ? -kInf : fac * mx;
          const bool grow = top > mf + kSlack;
          if (__any_sync(0xffffffffu, grow) || vnow != vmul) {
            if (vnow < 0.f) {
              vnow = -vnow;
              uint32_t nan_groups = 0;
#pragma unroll 1
              for (int u = 0; u < kTileUnits; u++) {
                // the unit's tokens [c0, c1)
                const uint32_t sees = ((1u << min(16, max(0, c1 - 16 * u))) - 1) & ~((1u << min(16, max(0, c0 - 16 * u))) - 1);
#pragma unroll
                for (int g = 0; g < NG; g++) nan_groups |= (s_nan[par][u][g] & sees) != 0 ? 1u << g : 0u;
              }
              s_nan_row[tid] |= (uint8_t)nan_groups;
            }
            const float shrink = vmul == 0.f ? 1.f : vnow / vmul;
            vmul = vnow;
            const float now = grow ? top : mf;
            const float f = mf == -kInf ? 1.f : exp2_fast(mf - now);
            mf = now;
            l *= f;
            if (j != j0) {
#pragma unroll 1
              for (int k = 0; k < HD; k += 32) {
                tmem_ld32(t_o + k, sv);
#pragma unroll
                for (int i = 0; i < 32; i++) sv[i] = __float_as_uint(__uint_as_float(sv[i]) * f * shrink);
                tmem_st32(t_o + k, sv);
              }
            }
          }
          const uint64_t fac2 = pack2(fac, fac), add2 = pack2(mf == -kInf ? 0.f : kLift - mf, mf == -kInf ? 0.f : kLift - mf);
          uint64_t l2 = 0;
#pragma unroll 1
          for (int k = 0; k < kTileTok; k += 32) {
            uint32_t pw[16];
            tmem_ld32(t_s + k, sv);
#pragma unroll
            for (int i = 0; i < 16; i++) {
              float e0, e1;
              unpack2(fma2((uint64_t)sv[2 * i] | (uint64_t)sv[2 * i + 1] << 32, fac2, add2), e0, e1);
              e0 = exp2_fast(e0);
              e1 = exp2_fast(e1);
              l2 = add2_f32(l2, pack2(e0, e1));
              pw[i] = bits(__floats2half2_rn(e0, e1));
            }
            tmem_st16(t_s + k / 2, pw);
          }
          {
            float e0, e1;
            unpack2(l2, e0, e1);
            l += e0 + e1;
          }
          tmem_wait_st();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[x]);
        }
      }
      n += n_here;
      w += n_here;
      stage += n_here;
      if (stage == it.stages) {
        stage = -kItemCost;
        if (w < w1) next_item();
      }
      // the scores have been read for the last time, so the next segment's can start beside what follows
      if (more()) load_queries();

      // ---- the segment's result ----
      const bool whole = n_here == at.stages, direct = whole && !split;
      const bool starts_here = item_at >= w0;
      float* mine = a.part + (size_t)(2 * blockIdx.x + starts_here) * kTileRows * (HD + 2);
      if (active) {
        wait(&o_full[x], nseg & 1);
        nseg++;
        tc_fence_after_sync();
      }
      if (active && rows) {
        // unscale comes second: beside very small or very large values its product with the other factor may not be a
        // normal number
        const float inv = direct ? (l == 0.f ? 0.f : 1.f / l) : kUnlift;
        const size_t out_row = (size_t)((at.r0 + q_row / a.group) * a.out_stride) + (size_t)(at.head * a.group + q_row % a.group) * HD;
#pragma unroll 1
        for (int k = 0; k < HD / 32; k++) {
          uint32_t sv[32];
          tmem_ld32(t_o + k * 32, sv);
          if (lrow < row_n) {
            float y[32];
#pragma unroll
            for (int h = 0; h < 2; h++)
#pragma unroll
              for (int i = 0; i < 16; i++) y[16 * h + 2 * (i % 8) + i / 8] = __uint_as_float(sv[16 * h + i]) * inv * unscale;
            if (l != l || (s_nan_row[tid] >> (k / T::kWpg) & 1)) {
#pragma unroll
              for (int i = 0; i < 32; i++) y[i] = __uint_as_float(0x7fc00000u);
            }
            if (direct) {
              uint16_t* o = static_cast<uint16_t*>(a.out) + out_row + k * 32;
#pragma unroll
              for (int i = 0; i < 32; i += 8) {
                uint32_t v[4];
#pragma unroll
                for (int e = 0; e < 4; e++)
                  v[e] = f32_to_bf16_rn(y[i + 2 * e]) | ((uint32_t)f32_to_bf16_rn(y[i + 2 * e + 1]) << 16);
                if (a.vec_out) {
                  *reinterpret_cast<uint4*>(o + i) = make_uint4(v[0], v[1], v[2], v[3]);
                } else {
#pragma unroll
                  for (int e = 0; e < 8; e++) o[i + e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
                }
              }
            } else {
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                __stcg(reinterpret_cast<float4*>(mine + (size_t)row * HD + k * 32 + i),
                       make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]));
            }
          }
        }
        tc_fence_before_sync();
      }
      if (!direct) {
        if (lrow < row_n)  // a half without work has seen nothing
          __stcg(reinterpret_cast<float2*>(mine + (size_t)kTileRows * HD + 2 * row), make_float2(mf, l * kUnlift));
        const int b0 = (int)(item_at / per), b1 = (int)((item_at + at.stages - 1) / per);
        __threadfence();
        named_sync(1, kSoftThreads);
        if (!whole) {
          if (tid == 0) {
            const int old = atomicAdd(a.count + b0, 1);
            s_last = old == b1 - b0;
            if (old == b1 - b0) atomicExch(a.count + b0, 0);
            __threadfence();
          }
          named_sync(1, kSoftThreads);
        }
        if (whole || s_last) {
          // a warp sums a row at a time, four rows and two parts in flight
          const int sides = split ? 2 : 1, parts = (b1 - b0 + 1) * sides;
          constexpr int kAcross = HD / 4, kStep = kSoftThreads / kAcross;
          const int d = tid % kAcross * 4;
          auto slot = [&](int k) { return a.part + (size_t)(2 * (b0 + k / sides) + (k / sides == 0)) * kTileRows * (HD + 2); };
          for (int r0 = tid / kAcross; r0 < row_n; r0 += 4 * kStep) {
            float mm[4], ll[4];
            float4 y[4];
#pragma unroll
            for (int q = 0; q < 4; q++) mm[q] = -kInf, ll[q] = 0.f, y[q] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
            for (int k = 0; k < parts; k++) {
              const float* p = slot(k);
              float2 ml[4];
              float4 v[4];
#pragma unroll
              for (int q = 0; q < 4; q++) {
                const int rr = min(r0 + q * kStep, row_n - 1) + (k % sides) * kHalf;
                ml[q] = __ldcg(reinterpret_cast<const float2*>(p + (size_t)kTileRows * HD + 2 * rr));
                v[q] = __ldcg(reinterpret_cast<const float4*>(p + (size_t)rr * HD + d));
              }
#pragma unroll
              for (int q = 0; q < 4; q++) {
                const float now = fmaxf(mm[q], ml[q].x);
                // never 0 for what has seen something, so that a value that is not a number stays one
                const float f = ml[q].y != ml[q].y ? 1.f : ml[q].x == -kInf ? 0.f : fmaxf(exp2_fast(ml[q].x - now), 0x1p-126f);
                const float g = ll[q] != ll[q] ? 1.f : mm[q] == -kInf ? 0.f : exp2_fast(mm[q] - now);
                mm[q] = now;
                ll[q] *= g;
                y[q].x *= g, y[q].y *= g, y[q].z *= g, y[q].w *= g;
                if (f != 0.f) {  // what a half without work did not write is not used
                  ll[q] = fmaf(ml[q].y, f, ll[q]);
                  y[q].x = fmaf(v[q].x, f, y[q].x), y[q].y = fmaf(v[q].y, f, y[q].y);
                  y[q].z = fmaf(v[q].z, f, y[q].z), y[q].w = fmaf(v[q].w, f, y[q].w);
                }
              }
            }
#pragma unroll
            for (int q = 0; q < 4; q++) {
              const int rr = r0 + q * kStep;
              if (rr >= row_n) continue;
              const float inv = ll[q] == 0.f ? 0.f : 1.f / ll[q];
              const long long qr = (long long)at.tile * kTileRows + rr;
              uint16_t* o = static_cast<uint16_t*>(a.out) + (size_t)((at.r0 + qr / a.group) * a.out_stride) +
                            (size_t)(at.head * a.group + qr % a.group) * HD + d;
              const uint32_t lo = f32_to_bf16_rn(y[q].x * inv) | ((uint32_t)f32_to_bf16_rn(y[q].y * inv) << 16);
              const uint32_t hi = f32_to_bf16_rn(y[q].z * inv) | ((uint32_t)f32_to_bf16_rn(y[q].w * inv) << 16);
              if (a.vec_out) {
                *reinterpret_cast<uint2*>(o) = make_uint2(lo, hi);
              } else {
                o[0] = (uint16_t)lo, o[1] = (uint16_t)(lo >> 16), o[2] = (uint16_t)hi, o[3] = (uint16_t)(hi >> 16);
              }
            }
          }
        }
        named_sync(1, kSoftThreads);
      }
    }
  }

  // every product and copy has been waited for: the softmax saw the last o_full, the converters the last copy
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == kWarpMma) tmem_dealloc(tmem, 512);
}

template <int HD, int NG>
int launch_one(coli_ctx* ctx, TileArgs& a) {
  using T = Tile<HD, NG>;
  const int grid = ctx->num_sms < kKvCounters ? ctx->num_sms : kKvCounters;
  static_assert((size_t)2 * kTileRows * (HD + 2) <= kKvPartFloats, "a CTA leaves more than there is room for");
  int rc = ensure_kv_part(ctx);
  if (rc != COLI_OK) return rc;
  a.part = ctx->d_kv_part;
  auto kern = kv4_tile_kernel<HD, NG>;
  static std::atomic<uint64_t> ready{0};  // devices (below 64) on which this instance has its attribute
  const uint64_t bit = ctx->device < 64 ? 1ull << ctx->device : 0;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem);
    if (e != cudaSuccess) return cuda_fail(ctx, e, "kv4_attention attribute");
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  ProfScope prof(ctx, COLI_KERNEL_ATTENTION);
  cudaError_t e = launch_k(kern, grid, kTileThreads, T::kSmem, ctx->stream, true, false, a);
  if (e != cudaSuccess) return cuda_fail(ctx, e, "kv4_attention launch");
  return COLI_OK;
}

}  // namespace

int launch_kv4_tiles(coli_ctx* ctx, const Kv4View& c, const Kv4Plan& p, const void* q, long long q_stride, int q_heads,
                     float scale, int window, void* out, long long out_stride) {
  TileArgs a{c, p, q, q_stride, q_heads / c.heads, scale, window, out, out_stride};
  a.vec = ((uintptr_t)q % 16 == 0) && q_stride % 8 == 0;
  a.vec_out = ((uintptr_t)out % 16 == 0) && out_stride % 8 == 0;
  a.count = ctx->d_kv_count;
  a.err = ctx->d_status;
  a.wait_ns = ctx->wait_ns ? ctx->wait_ns : kWaitLimitNs;
  a.withhold = ctx->test_withhold > 0;
  if (a.withhold) ctx->test_withhold--;
  if (c.hd == 64) return c.ng == 1 ? launch_one<64, 1>(ctx, a) : launch_one<64, 2>(ctx, a);
  return c.ng == 1 ? launch_one<128, 1>(ctx, a) : c.ng == 2 ? launch_one<128, 2>(ctx, a) : launch_one<128, 4>(ctx, a);
}

}  // namespace coli
