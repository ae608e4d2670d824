// y = resid + act(W x + bias) * mul with 16-bit weights (layout: dense.h), on the fifth-generation tensor cores.
//
// D = W X^T: the rows of W are the instruction's M (128, or 256 of a pair of CTAs), the tokens its N (16 to 256). Every SM (or pair)
// has one CTA and takes such tiles whole while there is one for each; what is left is split along the columns, so that one token
// keeps every SM streaming a run of W, and many tokens leave no part of a wave idle (dense_plan). A tile that several shares have
// a part of is joined by the one that arrives last, in the order of the shares, so results do not depend on who that is.
//
// One CTA, 20 warps: a producer (W by bulk copies, x by tiled ones, a ring of stages), a thread that issues the products, and
// sixteen warps for what follows (bias, activation, factor, residual), which take a tile from tensor memory while the next one
// is being formed in another part of it. The ring is filled with weights before the work ahead in the stream is waited for.
// Threads hold rows of W (128 neighbouring outputs of a token), so that rows of y at any alignment are read and written whole.
//
// Sums. The tensor core cuts a sum off where binary32 would round it, always towards zero: 6144 products lose some 2^-17 that
// way. Where y is binary32 chunks of kChunk column tiles are formed by themselves and added in registers (of 4096 tokens, 6144 x
// 6144, 195 us for 169; twice as long chunks lose twice as much for half of that; of binary32 activations chunks half as long lose half
// as much and take 3 to 15 % longer). Errors against 64 bits, in norm: 2.4e-7 for 6144
// columns of bf16 and of binary32 (7.7e-7 in tiles of 128 tokens and more); without chunks 1.2e-6 to 5e-6 (1.8e-5).
// Binary32 activations enter as parts of 8 bits by truncation, x = h + m + l exactly from 2^-110 on, to 2^-133 below (two parts, 16
// bits, where y is rounded to 8),
// each multiplied with the same staged tile of W. Where the parts' columns are 256 at most they are one instruction's, which reads
// the tile once (24 tokens, 6144 x 6144: 18.4 us against 21.1), and their sums are added by the last warps.
// Measured (us; W = O x I): one token, 6144 x 6144, residual 14.3 (5.3 TB/s, 0.78 of a copy's rate), f32 17.8; 24 tokens, 50021 x
// 6144, f32 logits 92 (6.7 TB/s, 0.98): bound by W's bytes, and at the small end by launch, first stages and the join of parts (4
// us). 301 f32 tokens, 2048 x 6144, silu and factor 32: L2 bytes, the join, and x laid out ahead. 4096 tokens, 6144 x 6144, gelu,
// bias, residual 211 (1465 TFLOP/s) over seconds, at the 1.47 GHz that the power limit leaves, the bare product 196, the library's 192;
// in short runs 187, 169 and 169. Tensor pipe active 82 % of the time.
// What it cost to find: factor and residual read where they are used, not a group ahead (prompt 348 us; 252 so); one CTA's 128 x
// 256 tiles, which ask L2 for 96 bytes a cycle and SM (219 us bare; pairs 183); 24 bytes of spilled registers inside the loop over
// chunks (480 us instead of 214: the ring leaves no first-level cache); even runs of many tiles for every
// share, so that W came from memory for each tile of tokens (2048 tokens, 20000 rows: 370 us, 273 so); precise exponentials, divisions and erfc (silu of 1748 x 20122:
// 120 us, 77 so). Dropped: setmaxnreg to give the last warps more registers (the producer spills), spare warps that lay out x
// stage by stage instead of a kernel ahead (f32 token 23.9 us against 18.3), tiles of 256 running sums (463 us), the parts of a
// tile all copied into the ring when it is joined (no faster: writing, the fence and the count take as long as reading).
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "dense.h"
#include "pipe.h"
#include "tc.h"

namespace coli {

namespace {

constexpr int kEpiWarps = 16, kWarpEpi = 4;  // warps 0 and 1: producer, products; a quarter of the lanes goes by warp % 4
constexpr int kThreads = (kWarpEpi + kEpiWarps) * 32;
constexpr int kChunk = 4;   // column tiles
constexpr int kGroup = 8;   // tokens that a thread of the last warps takes at a time
constexpr int kSets = kEpiWarps / 4;
static_assert(kSets == kDenseCounters, "a counter for each set");

// P parts of x for a staged tile of W. EXACT: y is binary32. PAIR: two CTAs of a cluster form 256 rows x N tokens with one
// instruction (cta_group::2), each staging its 128 rows and half of the tokens.
// The most tokens of a pair's tile: more running sums than 48 of a thread would not stay in registers.
template <bool EXACT>
constexpr int kPairTokens = EXACT ? 192 : 256;

template <int N, int P, bool EXACT, bool PAIR>
struct Shape {
  static constexpr int kCtas = PAIR ? 2 : 1;
  static constexpr int kXRows = N / kCtas;
  static constexpr uint32_t kX = P * kXRows * 128;
  static constexpr uint32_t kStage = kDenseTile + kX;
  static constexpr int kStages = std::min<uint32_t>(12, 224 * 1024 / kStage);
  static constexpr uint32_t kSmem = 1024 + kStages * kStage;
  // Parts side by side are one instruction's columns as long as those are enough: it reads W's tile once instead of P times, and
  // the small parts' sums lose nothing to the large ones'.
  static constexpr bool kWide = P > 1 && P * N <= 256;
  static constexpr int kCols = kWide ? P * N : N;
  // Accumulators. Chunks of few products are formed faster than a round trip between the two sides takes.
  static constexpr int kAcc = kCols <= 16 ? 16 : kCols <= 32 ? 32 : kCols <= 64 ? 64 : kCols <= 128 ? 128 : 256;  // columns apart
  static constexpr int kAccs = EXACT && kAcc <= 128 ? 4 : 2;
  static constexpr int kTmem = kAccs * kAcc;  // a power of two from 32 on
  static constexpr int kGroups = N / kGroup;
  static constexpr int kMine = EXACT ? (kGroups + kSets - 1) / kSets : 0;  // groups of a warp whose sums it holds
};

struct TileArgs {
  DenseArgs d;
  int kt, rt, nt;       // column tiles; tiles of 128 rows, or 256 of a pair; tiles of tokens
  int tail0;            // tiles up to this one are whole ones of a share: number `share`, then every `shares`-th
  int tail_shares;      // the shares of what is left
  long long tail_total; // its units
  bool stream;  // W is read once
  float* part;  // per CTA two of [N / 4][128][4]
  int* count;   // per CTA, zero between calls
  uint64_t wait_ns;
  bool withhold;  // test hook: the call's first copy is withheld, and the waits on it give up
};

// The numbers of tiles: groups of kBeside tiles of tokens (the last may be smaller), in each one row tile after another. What
// shares work on at a time is then a few rows and a few tokens: W passes memory once for a group, however large it is.
constexpr int kBeside = 8;
struct Place {
  int rows, tokens;  // tiles
};
__device__ __forceinline__ Place place_of(int tile, int rt, int nt) {
  const int g = tile / (rt * kBeside), i = tile - g * (rt * kBeside), width = max(1, min(kBeside, nt - g * kBeside)), rows = i / width;
  return Place{rows, g * kBeside + i - rows * width};
}

// A share's tiles, one after another.
struct Walk {
  int tile, k;  // the column tile from which on it is this share's

  __device__ __forceinline__ void next(const TileArgs& a, int shares, const Walk& tail) {
    k = 0;
    if (tile >= a.tail0) {
      tile++;
    } else {
      tile += shares;
      if (tile >= a.tail0) *this = tail;
    }
  }
};

__device__ __forceinline__ uint8_t* dense_at(uint8_t* w, int col_tiles, int o, int i) {
  const int r = o % kDenseRows, chunk = i % kDenseCols / 8;
  return w + ((size_t)(o / kDenseRows) * col_tiles + i / kDenseCols) * kDenseTile + r * 128 + ((chunk ^ (r & 7)) << 4);
}

__global__ void dense_pack_kernel(const uint16_t* src, int rows, int row0, int I, int col_tiles, uint8_t* w) {
  const long long chunks = (long long)((rows + kDenseRows - 1) / kDenseRows) * kDenseRows * col_tiles * 8;
  for (long long n = (long long)blockIdx.x * blockDim.x + threadIdx.x; n < chunks; n += (long long)gridDim.x * blockDim.x) {
    const int r = (int)(n / (col_tiles * 8)), i0 = (int)(n % (col_tiles * 8)) * 8;
    uint32_t v[4] = {0, 0, 0, 0};
    if (r < rows)
      for (int i = 0; i < 8; i++)
        if (i0 + i < I) v[i / 2] |= (uint32_t)src[(size_t)r * I + i0 + i] << (16 * (i & 1));
    *reinterpret_cast<uint4*>(dense_at(w, col_tiles, row0 + r, i0)) = make_uint4(v[0], v[1], v[2], v[3]);
  }
}

// Eight elements of x from `at` on, of which those from `have` on are 0.
__device__ __forceinline__ void dense_eight(const void* x, size_t at, int have, bool bf16, bool vec, float (&e)[8]) {
  if (bf16) {
#pragma unroll
    for (int i = 0; i < 8; i++) e[i] = i < have ? bf16_to_f32(__ldcg(static_cast<const unsigned short*>(x) + at + i)) : 0.f;
  } else if (vec && have >= 8) {
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const float4 q = __ldcg(reinterpret_cast<const float4*>(static_cast<const float*>(x) + at) + i);
      e[4 * i] = q.x, e[4 * i + 1] = q.y, e[4 * i + 2] = q.z, e[4 * i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) e[i] = i < have ? __ldcg(static_cast<const float*>(x) + at + i) : 0.f;
  }
}

// Them as P chunks of bf16: their parts of 8 bits. What is not finite stays what it is, in the first part alone.
template <int P>
__device__ __forceinline__ void dense_parts(float (&e)[8], uint32_t (&v)[P][4]) {
#pragma unroll
  for (int i = 0; i < 8; i++)
#pragma unroll
    for (int p = 0; p < P; p++) {
      const uint32_t u = __float_as_uint(e[i]);
      const bool finite = (u & 0x7f800000u) != 0x7f800000u;
      const uint32_t top = finite ? u & 0xffff0000u : (u & 0x7fffffu) ? 0x7fc00000u : u;
      v[p][i / 2] = i & 1 ? v[p][i / 2] | top : top >> 16;
      e[i] = finite ? e[i] - __uint_as_float(top) : 0.f;
    }
}

// x as P planes of bf16 rows that start at 16-byte boundaries.
template <bool BF16, int P>
__global__ void dense_x_kernel(const void* x, long long stride, int S, int I, bool vec, uint8_t* to) {
  griddep_launch_dependents();
  griddep_wait();
  const int chunks = (I + 7) / 8, n_all = S * chunks;  // at most 2^28
  for (int n = blockIdx.x * blockDim.x + threadIdx.x; n < n_all; n += gridDim.x * blockDim.x) {
    const int s = n / chunks, i0 = (n - s * chunks) * 8;
    float e[8];
    uint32_t v[P][4];
    dense_eight(x, (size_t)s * stride + i0, I - i0, BF16, vec, e);
    dense_parts<P>(e, v);
#pragma unroll
    for (int p = 0; p < P; p++)
      *reinterpret_cast<uint4*>(to + ((size_t)p * n_all + n) * 16) = make_uint4(v[p][0], v[p][1], v[p][2], v[p][3]);
  }
}

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float reciprocal_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

constexpr float kLog2e = 1.4426950408889634f;

// 1 / (1 + e^-x). A result that is rounded to 8 bits takes the exponential of an argument that rounds, off by about |x| units
// in the last place, and below 2^-126 is 0. EXACT: to a few units; e^-|x| = 2^t (1 + r ln 2), t + r the product -|x| log2(e) with
// what its rounding and the factor's lose.
template <bool EXACT>
__device__ __forceinline__ float dense_sigmoid(float x) {
  if constexpr (!EXACT) {
    return reciprocal_fast(1.f + exp2_fast(-x * kLog2e));
  } else {
    constexpr float kRest = (float)(1.4426950408889634074 - (double)kLog2e), kLn2 = 0.69314718f;
    const float a = fabsf(x) > 128.f ? 128.f : fabsf(x);  // NaN stays
    const float t = -a * kLog2e, r = fmaf(-a, kRest, fmaf(-a, kLog2e, -t));
    float e;
    asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(t));  // numbers below the normal ones stay
    e = fmaf(e, r * kLn2, e);
    const float s = reciprocal_fast(1.f + e);
    return x < 0.f ? e * s : s;
  }
}

// x/2 (1 + erf(x / sqrt 2)) = x/2 erfc(-x / sqrt 2), without cancellation on either side. erfc(a) = t 2^(P(t) - a^2 log2 e) for
// a >= 0 and t = 1 / (1 + a/2); P is a least-squares polynomial of degree 9 at 400 Chebyshev nodes of t for a up to 10.5, fitted
// to 40-digit values. Against those the whole is off by 3e-7 relative for a < 1 and 3e-7 a^2 above (binary32's rounding of the
// exponent).
__device__ __forceinline__ float dense_gelu(float x) {
  const float a = fabsf(x) * 0.70710678118654752f, t = reciprocal_fast(fmaf(0.5f, a, 1.f));
  float p = 0.21466025710105896f;
  p = fmaf(p, t, -1.0125515460968018f);
  p = fmaf(p, t, 1.740134835243225f);
  p = fmaf(p, t, -1.0993107557296753f);
  p = fmaf(p, t, -0.03750240430235863f);
  p = fmaf(p, t, -0.03969155624508858f);
  p = fmaf(p, t, 0.06400132924318314f);
  p = fmaf(p, t, 0.5548697113990784f);
  p = fmaf(p, t, 1.4410624504089355f);
  p = fmaf(p, t, -1.8256721496582031f);
  const float h = 0.5f * fabsf(x) * (t * exp2_fast(fmaf(a * a, -kLog2e, p)));
  if (x > 0.f) return x < __builtin_huge_valf() ? x - h : x;  // t is 0 of an infinity, and h not a number
  return -h;
}

template <bool EXACT, int N>
__device__ __forceinline__ void dense_act(float (&z)[N], int act) {
  switch (act) {
    case COLI_ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; i++) z[i] *= dense_sigmoid<EXACT>(z[i]);
      break;
    case COLI_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; i++) z[i] = dense_gelu(z[i]);
      break;
    case COLI_ACT_GELU_TANH:  // (1 + tanh u) / 2 = sigmoid(2 u)
#pragma unroll
      for (int i = 0; i < N; i++) z[i] *= dense_sigmoid<EXACT>(1.5957691216057308f * fmaf(0.044715f * z[i] * z[i], z[i], z[i]));
      break;
    case COLI_ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; i++) z[i] = z[i] < 0.f ? 0.f : z[i];
      break;
    case COLI_ACT_RELU2:
#pragma unroll
      for (int i = 0; i < N; i++) z[i] = z[i] < 0.f ? 0.f : z[i] * z[i];
      break;
  }
}

// Eight consecutive columns of this thread's lane (see tmem_ld16).
__device__ __forceinline__ void tmem_ld8(uint32_t at, float (&v)[8]) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(at)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; i++) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st8(uint32_t at, const float (&v)[8]) {
  uint32_t r[8];
#pragma unroll
  for (int i = 0; i < 8; i++) r[i] = __float_as_uint(v[i]);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(at)
               : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <int N, int P, bool EXACT, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) dense_kernel(const __grid_constant__ CUtensorMap x_map, const __grid_constant__ CUtensorMap w_map,
                                                            TileArgs a) {
  using H = Shape<N, P, EXACT, PAIR>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);  // [kStages][W tile | P tiles of x]
  // Of a pair, `full` and `acc_empty` of the first CTA count for both.
  __shared__ __align__(8) uint64_t full[H::kStages], empty[H::kStages], acc_full[H::kAccs], acc_empty[H::kAccs];
  __shared__ uint32_t s_tmem;
  __shared__ int s_last[kSets];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = PAIR ? (int)cluster_ctarank() : 0;
  const int shares = gridDim.x / H::kCtas, share = blockIdx.x / H::kCtas;
  griddep_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < H::kStages; i++) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < H::kAccs; i++) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], kEpiWarps * H::kCtas);
    }
    mbar_fence_init();
  }
  if (warp == 1) tmem_alloc_n<H::kCtas>(&s_tmem, H::kTmem);
  tc_fence_before_sync();
  if constexpr (PAIR)
    cluster_sync();
  else
    __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = s_tmem;

  // of what the whole tiles leave: units w0 to w1
  const long long w0 = a.tail_total * min(share, a.tail_shares) / a.tail_shares;
  const long long w1 = a.tail_total * min(share + 1, a.tail_shares) / a.tail_shares;
  const Walk tail{a.tail0 + (int)(w0 / a.kt), (int)(w0 % a.kt)}, start = a.tail0 ? Walk{share, 0} : tail;
  const uint32_t units = (uint32_t)(a.tail0 / shares * a.kt + (w1 - w0));
  bool alive = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (alive && !mbar_wait_suspend(bar, parity, a.wait_ns)) {
      set_error(a.d.err, COLI_E_TIMEOUT);
      alive = false;  // void from here on, but nothing hangs
    }
  };
  const bool holds = a.withhold && share == 0;  // the first copy, in both CTAs of a pair
  // The last arrivals on these barriers come before the CTA's memory goes, and with them the last reads of it. A parity tells a
  // phase from its neighbours alone: a thread that waits here has followed the barriers up to the fill before.
  auto wait_for_products = [&](uint32_t fills) {
    for (uint32_t i = fills > (uint32_t)H::kStages ? fills - H::kStages : 0; i < fills; i++)
      wait(&empty[i % H::kStages], (i / H::kStages) & 1);
  };

  if (warp == 0) {
    // ------------------------------------ producer ------------------------------------
    if (elect_one()) {
      const uint64_t once = l2_evict_first_policy();
      const uint32_t full0 = PAIR ? cluster_address(smem_u32(full), 0) : smem_u32(full);
      struct At {
        Walk walk;
        Place place;
      };
      auto advance = [&](At& at) {
        if (++at.walk.k < a.kt) return;
        at.walk.next(a, shares, tail);
        at.place = place_of(at.walk.tile, a.rt, a.nt);
      };
      At w_at{start, place_of(start.tile, a.rt, a.nt)}, x_at = w_at;
      auto copy_w = [&](uint32_t n) {
        const uint32_t s = n % H::kStages;
        uint8_t* to = smem + s * H::kStage;
        const int tile = (w_at.place.rows * H::kCtas + rank) * a.kt + w_at.walk.k;
        if (!(holds && n == 0)) {
          if (rank == 0) mbar_arrive_expect_tx(&full[s], H::kStage * H::kCtas);
          if constexpr (PAIR) {
            tma_load_2d_pair(to, &w_map, 0, tile * kDenseRows, full0 + s * 8);
          } else {
            const uint8_t* from = a.d.w + (size_t)tile * kDenseTile;
            if (a.stream)
              bulk_g2s_stream(to, from, kDenseTile, &full[s], once);
            else
              bulk_g2s(to, from, kDenseTile, &full[s]);
          }
        }
        advance(w_at);
      };
      auto copy_x = [&](uint32_t n) {
        const uint32_t s = n % H::kStages;
        if (!(holds && n == 0))
#pragma unroll
          for (int p = 0; p < P; p++) {
            uint8_t* to = smem + s * H::kStage + kDenseTile + p * H::kXRows * 128;
            const int y = p * a.d.S + x_at.place.tokens * N + rank * H::kXRows;
            if constexpr (PAIR)
              tma_load_2d_pair(to, &x_map, x_at.walk.k * kDenseCols, y, full0 + s * 8);
            else
              tma_load_2d(to, &x_map, x_at.walk.k * kDenseCols, y, &full[s]);
          }
        advance(x_at);
      };
      const uint32_t ahead = units < (uint32_t)H::kStages ? units : (uint32_t)H::kStages;
      for (uint32_t n = 0; n < ahead; n++) copy_w(n);  // weights do not depend on the work before this call
      griddep_wait();
      for (uint32_t n = 0; n < ahead; n++) copy_x(n);
      uint32_t n = ahead;
      for (; n < units && alive; n++) {
        wait(&empty[n % H::kStages], (n / H::kStages + 1) & 1);
        if (!alive) break;
        copy_w(n);
        copy_x(n);
      }
      // no copy is in flight when the CTA ends, whatever has been given up; of a pair the first CTA waits for both
      if (rank == 0)
        for (uint32_t i = n > (uint32_t)H::kStages ? n - H::kStages : 0; i < n; i++)
          if (!(holds && i == 0)) mbar_wait(&full[i % H::kStages], (i / H::kStages) & 1, a.wait_ns);
      // the second one's memory is read by products that the first CTA issues: its producer has seen every fill but the last
      if (rank == 1) wait_for_products(n);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------ products ------------------------------------
    // operands in uniform registers
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t w_desc = uniform(sw128_kmajor_desc(smem)), x_desc = uniform(sw128_kmajor_desc(smem + kDenseTile));
    if (rank == 0 && elect_one()) {
      constexpr uint32_t kId = bf16_f32_idesc(kDenseRows * H::kCtas, H::kCols);
      constexpr int kSteps = H::kWide ? 1 : P;
      uint32_t s = 0, phase = 0, chunk = 0, issued = 0;
      int left = (int)units;
      for (Walk walk = start; left > 0 && alive; walk.next(a, shares, tail)) {
        const int seg = min(a.kt - walk.k, left);
        for (int done = 0; done < seg && alive;) {
          const int here = EXACT ? min(kChunk, seg - done) : seg;
          wait(&acc_empty[chunk % H::kAccs], (chunk / H::kAccs + 1) & 1);
          tc_fence_after_sync();
          const uint32_t acc = tm + chunk % H::kAccs * H::kAcc;
          for (int i = 0; i < here; i++) {
            wait(&full[s], phase);
            if (!alive) break;  // nothing more is issued: what has been is waited for below, and the other side gives up by itself
            tc_fence_after_sync();
            const uint32_t at = s * (H::kStage >> 4);  // a descriptor's address field counts 16 bytes
#pragma unroll
            for (int p = kSteps - 1; p >= 0; p--)  // the small parts first
#pragma unroll
              for (int kk = 0; kk < 4; kk++)
                tc_mma_bf16_n<H::kCtas>(acc, w_desc + at + kk * 2, x_desc + at + p * (H::kXRows * 8) + kk * 2, kId,
                                        i > 0 || p < kSteps - 1 || kk > 0);
            tc_commit_n<H::kCtas>(&empty[s]);
            issued++;
            if (++s == (uint32_t)H::kStages) s = 0, phase ^= 1;
          }
          if (!alive) break;
          tc_commit_n<H::kCtas>(&acc_full[chunk % H::kAccs]);
          chunk++;
          done += here;
        }
        left -= seg;
      }
      alive = true;
      wait_for_products(issued);
      if (chunk > 0) wait(&acc_full[(chunk - 1) % H::kAccs], ((chunk - 1) / H::kAccs) & 1);
    }
    __syncwarp();
  } else if (warp >= kWarpEpi) {
    // ------------------------------------- what follows -------------------------------------
    griddep_wait();
    // the same in a warp, and visibly: what follows from it (tokens, their rows' addresses) stays out of the lanes
    const int set = EXACT ? (warp - kWarpEpi) >> 2 : __shfl_sync(0xffffffffu, (warp - kWarpEpi) >> 2, 0), row = (warp & 3) * 32 + lane;
    const uint32_t tm = tmem + ((uint32_t)(warp & 3) << 21);  // lanes 32 (warp % 4) on
    float broken = 0.f;  // not a number once a sum was not finite
    const uint32_t acc_empty0 = PAIR ? cluster_address(smem_u32(acc_empty), 0) : 0;
    auto free_acc = [&](uint32_t i) {
      if constexpr (PAIR)
        mbar_arrive_cluster(acc_empty0 + i * 8);
      else
        mbar_arrive(&acc_empty[i]);
    };
    // A tile's rows from this thread's, a group of tokens at a time. What is read beside the sums is asked for a group ahead. Many
    // tokens' arrays pass through L2 as the first to go, so that W and x stay (1748 x 1472 x 20122, silu, factor and residual:
    // 123 us without, 116 so).
    struct Beside {
      uint32_t f[kGroup], r[kGroup];
    };
    int o, t0;  // of the tile: this thread's row, the first token
    float bias;
    constexpr size_t kE = EXACT ? 4 : 2;
    auto ask = [&](Beside& v, int g) {
      if (g >= H::kGroups || o >= a.d.O) return;
      const int t = t0 + g * kGroup, n = a.d.S - t;
      const uint32_t off = (uint32_t)o * kE;
      auto load = [&](const void* p, long long stride, uint32_t (&to)[kGroup]) {
#pragma unroll
        for (int i = 0; i < kGroup; i++) {
          const char* at = static_cast<const char*>(p) + (t + i) * stride * kE + off;
          using T = std::conditional_t<EXACT, unsigned int, unsigned short>;
          if (i < n) to[i] = PAIR ? __ldcs(reinterpret_cast<const T*>(at)) : __ldcg(reinterpret_cast<const T*>(at));
        }
      };
      if (a.d.mul) load(a.d.mul, a.d.mul_stride, v.f);
      if (a.d.resid) load(a.d.resid, a.d.resid_stride, v.r);
    };
    auto value = [](uint32_t u) { return __uint_as_float(EXACT ? u : u << 16); };
    auto finish = [&](float (&sum)[kGroup], const Beside& v, int g) {
      if (o >= a.d.O) return;
      const int t = t0 + g * kGroup, n = a.d.S - t;
      const uint32_t off = (uint32_t)o * kE;
      float z[kGroup];
#pragma unroll
      for (int i = 0; i < kGroup; i++) {
        if (i < n) broken = fmaf(sum[i], 0.f, broken);
        z[i] = sum[i] + bias;
      }
      dense_act<EXACT>(z, a.d.act);
      if (a.d.mul)
#pragma unroll
        for (int i = 0; i < kGroup; i++) z[i] *= value(v.f[i]);
      if (a.d.resid)
#pragma unroll
        for (int i = 0; i < kGroup; i++) z[i] += value(v.r[i]);
#pragma unroll
      for (int i = 0; i < kGroup; i++) {
        char* at = static_cast<char*>(a.d.y) + (t + i) * a.d.y_stride * kE + off;
        using T = std::conditional_t<EXACT, float, unsigned short>;
        T v;
        if constexpr (EXACT)
          v = z[i];
        else
          v = __bfloat16_as_ushort(__float2bfloat16_rn(z[i]));
        if (i < n) {
          if constexpr (PAIR)
            __stcs(reinterpret_cast<T*>(at), v);
          else
            *reinterpret_cast<T*>(at) = v;
        }
      }
    };
    auto at_tile = [&](int tile) {
      const Place at = place_of(tile, a.rt, a.nt);
      o = (at.rows * H::kCtas + rank) * kDenseRows + row;
      t0 = at.tokens * N;
      bias = a.d.bias && o < a.d.O ? __ldcg(a.d.bias + o) : 0.f;
    };
    // the columns of a group's first part; those of the others are kXRows apart, and of a pair the second CTA's tokens behind all
    auto column = [&](uint32_t acc, int g) { return acc + g * kGroup + (H::kWide ? g * kGroup / H::kXRows * (P - 1) * H::kXRows : 0); };
    auto read_parts = [&](uint32_t acc, int g, float (&z)[kGroup]) {
      const uint32_t at = column(acc, g);
      tmem_ld8(at + (H::kWide ? P - 1 : 0) * H::kXRows, z);
      if constexpr (H::kWide) {
#pragma unroll
        for (int p = P - 2; p >= 0; p--) {
          float v[kGroup];
          tmem_ld8(at + p * H::kXRows, v);
#pragma unroll
          for (int i = 0; i < kGroup; i++) z[i] += v[i];
        }
      }
    };
    auto read_sums = [&](uint32_t acc, int g, float (&z)[kGroup]) {
      if constexpr (EXACT)
        tmem_ld8(column(acc, g), z);  // put there chunk by chunk
      else
        read_parts(acc, g, z);
    };
    uint32_t chunk = 0;
    int left = (int)units;
    for (Walk walk = start; left > 0; walk.next(a, shares, tail)) {
      const int tile = walk.tile, seg = min(a.kt - walk.k, left);
      const bool whole = seg == a.kt;
      Beside next;
      if constexpr (EXACT) {
        float sum[H::kMine][kGroup] = {};
#pragma unroll 1
        for (int done = 0; done < seg; done += kChunk) {
          wait(&acc_full[chunk % H::kAccs], chunk / H::kAccs & 1);
          __syncwarp();
          tc_fence_after_sync();
          const uint32_t acc = tm + chunk % H::kAccs * H::kAcc;
          const bool last = done + kChunk >= seg;
          if (!H::kWide && last && done == 0) break;  // one chunk: it is where it is read from below
#pragma unroll
          for (int m = 0; m < H::kMine; m++) {
            const int g = kSets * m + set;
            if (g >= H::kGroups) break;
            float v[kGroup];
            read_parts(acc, g, v);
#pragma unroll
            for (int i = 0; i < kGroup; i++) sum[m][i] += v[i];
            if (last) tmem_st8(column(acc, g), sum[m]);
          }
          if (last) break;
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) free_acc(chunk % H::kAccs);
          chunk++;
        }
        tmem_wait_st();
        at_tile(tile);
        if (whole) ask(next, set);
      } else {
        at_tile(tile);
        if (whole) ask(next, set);
        wait(&acc_full[chunk % H::kAccs], chunk / H::kAccs & 1);
        __syncwarp();
        tc_fence_after_sync();
      }
      const uint32_t acc = tm + chunk % H::kAccs * H::kAcc;
      if (whole) {
#pragma unroll 1
        for (int g = set; g < H::kGroups; g += kSets) {
          float z[kGroup];
          read_sums(acc, g, z);
          const Beside now = next;
          ask(next, g + kSets);
          finish(z, now, g);
        }
      } else {
        // a tile's beginning goes to the CTA's second part, a continuation to its first; four tokens of a row together
        constexpr size_t kPart = (size_t)(N / 4) * kDenseRows;
        float4* parts = reinterpret_cast<float4*>(a.part) + row;
        float4* mine = parts + ((size_t)2 * blockIdx.x + (walk.k == 0)) * kPart;
#pragma unroll 1
        for (int g = set; g < H::kGroups; g += kSets) {
          float z[kGroup];
          read_sums(acc, g, z);
#pragma unroll
          for (int i = 0; i < 2; i++) __stcg(mine + (g * 2 + i) * kDenseRows, make_float4(z[4 * i], z[4 * i + 1], z[4 * i + 2], z[4 * i + 3]));
        }
        // the shares of this tile: from the one that begins it to the one that ends it. The four warps of a set, which hold
        // all rows of their tokens, join them on their own.
        const long long u0 = (long long)(tile - a.tail0) * a.kt, u1 = u0 + a.kt - 1;
        const int first = (int)(((u0 + 1) * a.tail_shares - 1) / a.tail_total), last = (int)(((u1 + 1) * a.tail_shares - 1) / a.tail_total);
        __threadfence();
        named_sync(1 + set, 128);
        if ((tid & 127) == 0) {
          int* count = a.count + (first * H::kCtas + rank) * kSets + set;
          s_last[set] = atomicAdd(count, 1) == last - first;
          if (s_last[set]) *count = 0;
        }
        named_sync(1 + set, 128);
        if (s_last[set]) {
          __threadfence();
          // in CTA order, its own sums from tensor memory; the first of the others' is asked for a group ahead, too
          const int own = (int)share, other = first == own ? first + 1 : first;
          auto part_of = [&](int c, int g, int i) { return __ldcg(parts + ((size_t)2 * (c * H::kCtas + rank) + (c == first)) * kPart + (g * 2 + i) * kDenseRows); };
          float4 p[2];
          auto ask_part = [&](int g) {
            if (g < H::kGroups)
#pragma unroll
              for (int i = 0; i < 2; i++) p[i] = part_of(other, g, i);
          };
          ask_part(set);
          ask(next, set);
#pragma unroll 1
          for (int g = set; g < H::kGroups; g += kSets) {
            float mine8[kGroup], z[kGroup];
            read_sums(acc, g, mine8);
#pragma unroll
            for (int i = 0; i < 2; i++) z[4 * i] = p[i].x, z[4 * i + 1] = p[i].y, z[4 * i + 2] = p[i].z, z[4 * i + 3] = p[i].w;
            if (first == own)
#pragma unroll
              for (int i = 0; i < kGroup; i++) z[i] += mine8[i];  // two terms: in either order the same
            ask_part(g + kSets);
            const Beside now = next;
            ask(next, g + kSets);
#pragma unroll 4
            for (int c = other + 1; c <= last; c++) {
              float4 v[2];
              if (c != own)
#pragma unroll
                for (int i = 0; i < 2; i++) v[i] = part_of(c, g, i);
              else
#pragma unroll
                for (int i = 0; i < 2; i++) v[i] = make_float4(mine8[4 * i], mine8[4 * i + 1], mine8[4 * i + 2], mine8[4 * i + 3]);
#pragma unroll
              for (int i = 0; i < 2; i++) z[4 * i] += v[i].x, z[4 * i + 1] += v[i].y, z[4 * i + 2] += v[i].z, z[4 * i + 3] += v[i].w;
            }
            finish(z, now, g);
          }
        }
        named_sync(1 + set, 128);  // s_last is read before it is written again
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) free_acc(chunk % H::kAccs);
      chunk++;
      left -= seg;
    }
    if (broken != 0.f) set_error(a.d.err, COLI_E_NONFINITE);
  }
  tc_fence_before_sync();
  if constexpr (PAIR)
    cluster_sync();
  else
    __syncthreads();
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc_n<H::kCtas>(tmem, H::kTmem);
}

// A call's tiles and how they are dealt out: what takes the fewest cycles by a model that was fitted to 12274 measurements (O, I
// of 768 to 50021, S of 1 to 4096, each type; what it picks takes 1.5 to 1.8 % more than the best of them on average, 19 % at most).
//   A column tile takes its bytes from L2 at 64 a cycle and 60, or its products and 60; a tile 220 more. W is read at 26 bytes a
//   cycle and SM, of which two thirds are enough, and eight tenths of it once more for each further tile of tokens. A split tile
//   takes N times 40 cycles and 19.6 for each part, or 3.5 more where shares begin anywhere (their ends meet two tiles). A pair of
//   CTAs, which halves the tokens' bytes, 2100.
// Tiles are dealt out whole as long as there is one for every share. What is left is split evenly over all shares (together with
// the last whole ones, or by itself), or each tile over as many shares q as there are for it. Measured, us, even shares of
// everything and as chosen: one token, 6144 x 6144, 15.2 14.1; 301 tokens there 33.7 24.4; 512 tokens, O = I = 4096, 23.2 18.4; 4096
// tokens, 6144 x 6144, 197 171; 2048 tokens, 20000 x 6144, 370 280 (even runs of many tiles read W from memory again and again).
struct Plan {
  int tokens;  // of a tile
  bool pair;
  int whole;   // tiles that each share takes whole
  int q;       // shares of each other tile, 0: all shares of all of them
};

Plan dense_plan(int S, int O, int I, int parts, bool exact, int num_sms) {
  const int most = exact ? kPairTokens<true> : kPairTokens<false>;
  const Plan all[] = {{16, false}, {32, false}, {64, false}, {128, false}, {64, true}, {128, true}, {most, true}};
  const int kt = (I + kDenseCols - 1) / kDenseCols;
  const double bytes = (double)dense_bytes(O, I);
  Plan best{};
  double least = 0;
  for (const Plan& p : all) {
    if ((p.tokens == 16) != (S <= 16)) continue;
    const int ctas = p.pair ? 2 : 1, N = p.tokens, shares = num_sms / ctas;
    const int nt = (S + N - 1) / N;
    const int tiles = (O + kDenseRows * ctas - 1) / (kDenseRows * ctas) * nt, waves = tiles / shares;
    const double unit = std::max((kDenseTile + parts * N / ctas * 128.0) / 64 + 60, parts * N * 2.0 + 60), tile = kt * unit + 220;
    const double read = bytes / (26.0 * num_sms) * (1 + 0.8 * (nt - 1)) / tiles;  // W for a tile, where all SMs read
    auto look = [&](int whole, int q) {
      const int rest = tiles - whole * shares;
      const long long used = q ? (long long)rest * q : std::min<long long>(shares, (long long)rest * kt);
      double cycles = std::max(tile, read * shares) * whole + (p.pair ? 2100 : 0);
      if (rest > 0) {
        const double each = q ? (double)((kt + q - 1) / q) / kt : (double)rest / used;  // tiles of a share
        cycles += std::max(tile * each, read * rest / std::min(1.0, used / (0.66 * shares)));
        if (q != 1 && !(q == 0 && rest % shares == 0)) cycles += N * (40 + 19.6 * (q ? q : 3.5 + std::max(1, (shares + rest - 1) / rest)));
      }
      if (least == 0 || cycles < least) least = cycles, best = Plan{p.tokens, p.pair, whole, q};
    };
    look(std::max(0, waves - 1), 0);
    const int rest = tiles - waves * shares;
    if (rest == 0) {
      look(waves, 1);
      continue;
    }
    if (waves) look(waves, 0);
    const int q_most = std::min(shares / rest, kt);
    for (int u = (kt + q_most - 1) / q_most, q = q_most;; u += (u + 3) / 4) {  // a share's column tiles
      q = (kt + u - 1) / u;
      look(waves, q);
      if (q == 1) break;
    }
  }
  return best;
}

template <int N, int P, bool EXACT, bool PAIR>
int launch_one(coli_ctx* ctx, TileArgs& a, const Plan& plan, const CUtensorMap& x_map, const CUtensorMap& w_map) {
  using H = Shape<N, P, EXACT, PAIR>;
  static_assert((size_t)2 * N * kDenseRows <= kPartFloats, "a CTA leaves more than there is room for");
  a.kt = (a.d.I + kDenseCols - 1) / kDenseCols;
  const int rows = kDenseRows * H::kCtas;
  a.nt = (a.d.S + N - 1) / N;
  a.rt = (a.d.O + rows - 1) / rows;
  a.stream = a.nt == 1;
  const int all = ctx->num_sms / H::kCtas, rest = a.rt * a.nt - plan.whole * all;
  a.tail0 = plan.whole * all;
  a.tail_total = (long long)rest * a.kt;
  a.tail_shares = plan.q ? std::max(1, rest * plan.q) : (int)std::min<long long>(all, a.tail_total);
  const int shares = plan.whole ? all : a.tail_shares;
  auto kern = dense_kernel<N, P, EXACT, PAIR>;
  static std::atomic<uint64_t> ready{0};  // devices (below 64) on which this instance has its attribute
  const uint64_t bit = ctx->device < 64 ? 1ull << ctx->device : 0;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, H::kSmem);
    if (e != cudaSuccess) return cuda_fail(ctx, e, "dense_linear attribute");
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(shares * H::kCtas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = H::kSmem;
  cfg.stream = ctx->stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = H::kCtas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 2 : 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, x_map, w_map, a);
  if (e != cudaSuccess) return cuda_fail(ctx, e, "dense_linear launch");
  return COLI_OK;
}

template <bool BF16, int P>
cudaError_t lay_out(coli_ctx* ctx, const DenseArgs& a, bool vec, uint8_t* to) {
  const long long chunks = (long long)a.S * ((a.I + 7) / 8);
  const int grid = (int)std::min<long long>((chunks + 127) / 128, (long long)ctx->num_sms * 16);
  return launch_k(dense_x_kernel<BF16, P>, grid, 128, 0, ctx->stream, true, false, a.x, a.x_stride, a.S, a.I, vec, to);
}

}  // namespace

cudaError_t launch_dense_pack(cudaStream_t stream, const uint16_t* src, int rows, int row0, int I, uint8_t* w) {
  dense_pack_kernel<<<1216, 256, 0, stream>>>(src, rows, row0, I, (I + kDenseCols - 1) / kDenseCols, w);
  return cudaGetLastError();
}

int launch_dense(coli_ctx* ctx, const DenseArgs& args, const CUtensorMap& w_map, int x_dtype, int y_dtype) {
  TileArgs a{};
  a.d = args;
  a.d.err = ctx->d_status;
  a.wait_ns = ctx->wait_ns ? ctx->wait_ns : kWaitLimitNs;
  a.withhold = ctx->test_withhold > 0;
  int rc = ensure_part(ctx);
  if (rc != COLI_OK) return rc;
  a.part = ctx->d_part;
  a.count = ctx->d_dense_count;
  const bool exact = y_dtype == COLI_DTYPE_F32;
  const int parts = x_dtype == COLI_DTYPE_BF16 ? 1 : !exact ? 2 : 3;
  // rows of x by tiled copies where they lie, or from planes laid out in the workspace
  const long long row = a.d.S == 1 ? (a.d.I + 7) / 8 * 8 : a.d.x_stride;
  const bool direct = parts == 1 && (uintptr_t)a.d.x % 16 == 0 && row % 8 == 0;
  const int S = a.d.S;
  const Plan t = dense_plan(S, a.d.O, a.d.I, parts, exact, ctx->num_sms);
  const int box = t.pair ? t.tokens / 2 : t.tokens;
  CUtensorMap map{};
  if (direct) {
    rc = encode_rows_map(ctx, &map, const_cast<void*>(a.d.x), S, a.d.I, row, kDenseCols, box, true);
  } else {
    rc = ensure_workspace(ctx, dense_x_bytes(S, a.d.I, parts));
    if (rc == COLI_OK) rc = encode_rows_map(ctx, &map, ctx->ws.base, (long long)parts * S, a.d.I, (a.d.I + 7) / 8 * 8, kDenseCols, box, true);
  }
  if (rc != COLI_OK) return rc;
  if (a.withhold) ctx->test_withhold--;
  ProfScope prof(ctx, COLI_KERNEL_LINEAR);
  if (!direct) {
    uint8_t* to = reinterpret_cast<uint8_t*>(ctx->ws.base);
    const bool vec = (uintptr_t)a.d.x % 16 == 0 && row % 4 == 0;
    const cudaError_t e = parts == 1   ? lay_out<true, 1>(ctx, a.d, false, to)
                          : parts == 2 ? lay_out<false, 2>(ctx, a.d, vec, to)
                                       : lay_out<false, 3>(ctx, a.d, vec, to);
    if (e != cudaSuccess) return cuda_fail(ctx, e, "dense_linear layout launch");
  }
  auto tokens = [&](auto p, auto y32) {
    constexpr int P = decltype(p)::value;
    constexpr bool E = decltype(y32)::value;
    if (t.pair) {
      if (t.tokens == 64) return launch_one<64, P, E, true>(ctx, a, t, map, w_map);
      if (t.tokens == 128) return launch_one<128, P, E, true>(ctx, a, t, map, w_map);
      return launch_one<kPairTokens<E>, P, E, true>(ctx, a, t, map, w_map);
    }
    if (t.tokens == 16) return launch_one<16, P, E, false>(ctx, a, t, map, w_map);
    if (t.tokens == 32) return launch_one<32, P, E, false>(ctx, a, t, map, w_map);
    if (t.tokens == 64) return launch_one<64, P, E, false>(ctx, a, t, map, w_map);
    return launch_one<128, P, E, false>(ctx, a, t, map, w_map);
  };
  if (parts == 3) return tokens(std::integral_constant<int, 3>{}, std::true_type{});
  if (parts == 2) return tokens(std::integral_constant<int, 2>{}, std::false_type{});
  if (exact) return tokens(std::integral_constant<int, 1>{}, std::true_type{});
  return tokens(std::integral_constant<int, 1>{}, std::false_type{});
}

}  // namespace coli
