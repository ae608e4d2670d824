// Log probabilities: a row's log-sum-exp, entropy and largest entries in one pass over its logits.
//
// Bound by memory: every logit is read once. A CTA takes a row, or a part of one where there are few rows; the last CTA of a
// row to arrive joins the parts, in their order. A thread keeps s = sum e^(x - b) and t = sum (x - b) e^(x - b) (entropy =
// log s - t / s, relative to the base b) for two streams of entries at a time, which the packed instructions take together. The
// base follows the largest entry with a slack of 2^16, so that it hardly ever moves.
//
// The largest entries cost the pass nothing but the place of each thread's maximum. An entry's key is its value with its index
// below, so keys never tie and the lower index wins. The maxima of 64 groups of threads are 64 entries, so the k-th largest of
// them is a bound that k entries reach at least; only entries of threads whose own maximum reaches it are looked through again
// (out of L2, all threads together), and what is found, about k ln k entries, is ranked by comparison with one another.
// Where ties make it more than there is room for, the k-th largest of those found is a higher bound of the same kind, and the
// search repeats.
//
// Measured: 2048 rows of 65536 (f32, one alternative) 89 us, 6.0 TB/s, 0.89 of a copy's rate (0.95 without alternatives, 114 us
// with 20: their entries come from memory again); 64 rows of 151001 (bf16, 20 alternatives, 9 CTAs a row) 14.2 us, 9.4 without
// alternatives: a chain of round trips to L2 (entries, parts written, counted, read) and barriers; one row of 50021 6.8 us, 4.2
// without. A vector on its way in registers instead of shared memory held the f32 rows to 4.1 TB/s (143 us); a maximum that moves with every larger entry, 151 us
// then; threads that look through their own entries alone, 290 us with 20 alternatives; bounds from 32 groups, four times the
// entries to rank for 32 alternatives.
#include "logprobs.h"
#include "pipe.h"

namespace coli {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRoom = kLogprobMostParts * COLI_MAX_TOP;  // entries that reach the bound
constexpr int kLooks = 2;    // vectors that a thread looks through together
constexpr int kFlight = 7;   // vectors of a thread on their way
// Vectors of a thread that are not worth another CTA of the row: they are on their way together, and fewer parts are joined
// sooner (15 rows of 32003, 32 alternatives: 9.2 us with 4, 12.5 with 1).
constexpr int kFew = 4;
constexpr int kGroups = 64, kPerGroup = kThreads / kGroups;  // groups of threads whose maxima make the bound
constexpr float kInf = __builtin_huge_valf();
constexpr float kLowest = -3.402823466e38f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// 2^y is 0 in binary32 below this, and y 2^y then too
constexpr float kNothing = -300.f;
constexpr float kSlack = 16.f;  // by which an entry may pass the base, in powers of two

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float max_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}

__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}
// Arithmetic on two binary32 values in a register pair.
__device__ __forceinline__ uint64_t pack2(float x, float y) { return (uint64_t)__float_as_uint(x) | (uint64_t)__float_as_uint(y) << 32; }
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  return r;
}
__device__ __forceinline__ float low(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float high(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

// Keys: whole numbers in the order of (value, then lower index). Zeros of both signs are the same value.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u >> 31) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t key_of(float x, int index) { return (uint64_t)ordered(x) << 32 | (0xffffffffu - (uint32_t)index); }
__device__ __forceinline__ int index_of(uint64_t key) { return (int)(0xffffffffu - (uint32_t)key); }
__device__ __forceinline__ float value_of(uint64_t key) {
  const uint32_t u = (uint32_t)(key >> 32);
  return __uint_as_float((u >> 31) ? u & 0x7fffffffu : ~u);
}
// Above every key of -infinity, which is no alternative; not above any other.
constexpr uint64_t kLeast = (uint64_t)0x00800000u << 32;

// Sums over a set of entries relative to a base b, -infinity where there is none yet.
struct Sums {
  float b, s, t;
  // where differences are taken from: finite, so that entries of -infinity add nothing
  static __device__ __forceinline__ float from(float b) { return fmaxf(b, kLowest); }
  // what carries sums over from base b to `to`, which is no smaller; c = scale log2 e
  static __device__ __forceinline__ float shift(float b, float to, float c) { return max_nan((from(b) - from(to)) * c, kNothing); }
  __device__ __forceinline__ void move(float to, float c) {
    const float y = shift(b, to, c), f = exp2_fast(y);
    t = f * fmaf(s, y, t);
    s *= f;
    b = to;
  }
  __device__ __forceinline__ void join(Sums o, float c) {
    const float to = fmaxf(b, o.b);
    move(to, c);
    o.move(to, c);
    s += o.s;
    t += o.t;
  }
};

// The sums of a thread, over the even and the odd entries of its vectors.
template <int E>
struct Stream {
  float b = -kInf, limit = -kInf;
  uint64_t minus = pack2(-kLowest, -kLowest), s = 0, t = 0;

  __device__ __forceinline__ void add(const float (&x)[E], float top, float c, float slack) {
    if (top > limit) {
      const float y = Sums::shift(b, top, c), f = exp2_fast(y);
      t = mul2(fma2(s, pack2(y, y), t), pack2(f, f));
      s = mul2(s, pack2(f, f));
      b = top;
      limit = top + slack;
      minus = pack2(-Sums::from(top), -Sums::from(top));
    }
    const uint64_t cc = pack2(c, c);
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const uint64_t d = mul2(add2(pack2(x[i], x[i + 1]), minus), cc);
      const uint64_t y = pack2(max_nan(low(d), kNothing), max_nan(high(d), kNothing));
      const uint64_t e = pack2(exp2_fast(low(y)), exp2_fast(high(y)));
      s = add2(s, e);
      t = fma2(e, y, t);
    }
  }
  __device__ __forceinline__ Sums sums() const { return Sums{b, low(s) + high(s), low(t) + high(t)}; }
};

template <bool BF16>
struct Row {
  static constexpr int E = BF16 ? 8 : 4;  // elements of a vector
  const char* at;                         // the boundary at or before the row's first element
  int shift, V;
  int whole0, wholes;  // the first vector that lies within the row, and how many do

  __device__ __forceinline__ bool is_whole(int j) const { return (unsigned)(j - whole0) < (unsigned)wholes; }
  // vector j; elements outside the row are -infinity
  __device__ __forceinline__ uint4 load(int j) const {
    const char* p = at + (size_t)j * 16;
    if (is_whole(j)) return __ldcg(reinterpret_cast<const uint4*>(p));
    const int e0 = j * E - shift;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      if constexpr (BF16) {
        auto half = [&](int h) -> uint32_t {
          const int e = e0 + 2 * i + h;
          return e >= 0 && e < V ? __ldcg(reinterpret_cast<const unsigned short*>(p) + 2 * i + h) : 0xff80u;
        };
        w[i] = half(0) | half(1) << 16;
      } else {
        const int e = e0 + i;
        w[i] = e >= 0 && e < V ? __ldcg(reinterpret_cast<const unsigned int*>(p) + i) : 0xff800000u;
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ void unpack(const uint4& r, float (&v)[E]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      if constexpr (BF16)
        v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      else
        v[i] = __uint_as_float(w[i]);
    }
  }
  __device__ __forceinline__ float one(int e) const {
    if constexpr (BF16)
      return bf16_to_f32(__ldcg(reinterpret_cast<const unsigned short*>(at) + shift + e));
    else
      return __ldcg(reinterpret_cast<const float*>(at) + shift + e);
  }
};

// 16 bytes into shared memory, waited for by groups: the copies on their way take no registers.
__device__ __forceinline__ void copy_async(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }

struct Shared {
  uint4 ring[kFlight][kThreads];  // each thread's vectors on their way
  Sums sums[kWarps];
  float most[kWarps];
  uint64_t group[kGroups];
  uint64_t found[kRoom];
  uint64_t best[COLI_MAX_TOP];
  uint64_t bound;
  int n, hits;
  bool last;
  uint16_t hit[kThreads];  // threads whose largest entry reaches the bound
};

// The k-th largest of s.group (no two alike, but for 0), or kLeast if that is none or less. s.bound holds kLeast when all threads
// come here, after a barrier.
__device__ __forceinline__ uint64_t find_bound(Shared& s, int k) {
  const uint64_t mine = s.group[threadIdx.x / kPerGroup];
  int above = 0;
#pragma unroll
  for (int j = 0; j < kGroups; j += kPerGroup) above += s.group[j + threadIdx.x % kPerGroup] > mine;
#pragma unroll
  for (int o = 1; o < kPerGroup; o *= 2) above += __shfl_xor_sync(0xffffffffu, above, o);
  if (threadIdx.x % kPerGroup == 0 && above == k - 1) s.bound = max64(mine, kLeast);
  __syncthreads();
  return s.bound;
}

// A group of threads gives its largest key.
__device__ __forceinline__ void give_group(Shared& s, uint64_t key) {
#pragma unroll
  for (int o = 1; o < kPerGroup; o *= 2) key = max64(key, __shfl_xor_sync(0xffffffffu, key, o));
  if (threadIdx.x % kPerGroup == 0) s.group[threadIdx.x / kPerGroup] = key;
}

// The k largest of the keys s.found[0..n), in order, into s.best; 0 behind them. All of the CTA's threads, between barriers.
__device__ __forceinline__ void rank_found(Shared& s, int n, int k) {
  const int tid = threadIdx.x;
  constexpr int kEach = kRoom / kThreads;
  // Many: the k-th largest of the groups' maxima is a bound again, and what is below it goes. More than kThreads keys give each
  // of the kGroups groups kPerGroup of them at least, and k groups stay at most.
  while (n > kThreads) {
    uint64_t mine[kEach], most = 0;
#pragma unroll
    for (int u = 0; u < kEach; u++) {
      mine[u] = tid + u * kThreads < n ? s.found[tid + u * kThreads] : 0;
      most = max64(most, mine[u]);
    }
    give_group(s, most);
    if (tid == 0) s.n = 0, s.bound = kLeast;
    __syncthreads();
    const uint64_t bound = find_bound(s, k);
#pragma unroll
    for (int u = 0; u < kEach; u++)
      if (mine[u] >= bound) s.found[atomicAdd(&s.n, 1)] = mine[u];
    __syncthreads();
    n = s.n;
    __syncthreads();
  }
  // Ranks are below n: what is cleared here and what is stored below are different entries, whichever warp comes first.
  if (tid >= n && tid < COLI_MAX_TOP) s.best[tid] = 0;
  for (int i0 = 0; i0 < n; i0 += kGroups) {
    const int i = i0 + tid / kPerGroup;
    const uint64_t mine = i < n ? s.found[i] : 0;
    int above = 0;
#pragma unroll 4
    for (int j = tid % kPerGroup; j < n; j += kPerGroup) above += s.found[j] > mine;
#pragma unroll
    for (int o = 1; o < kPerGroup; o *= 2) above += __shfl_xor_sync(0xffffffffu, above, o);
    if (i < n && above < k) s.best[above] = mine;
  }
  __syncthreads();
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, kLogprobCtas) logprob_kernel(LogprobArgs a) {
  constexpr int E = Row<BF16>::E;
  __shared__ Shared s;
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row_id = blockIdx.x / a.parts, part_id = blockIdx.x - row_id * a.parts;
  Row<BF16> row;
  row.V = a.V;
  row.shift = (int)(((uint64_t)row_id * (uint64_t)a.stride + a.shift_step) % E);
  row.at = static_cast<const char*>(a.x) + ((long long)row_id * a.stride - row.shift) * (BF16 ? 2 : 4);
  const int vecs = (a.V + row.shift + E - 1) / E;
  row.whole0 = row.shift > 0;
  row.wholes = max((a.V + row.shift) / E - row.whole0, 0);
  const int v0 = part_id * a.per, v1 = min(vecs, v0 + a.per);
  const float c = a.scale * kLog2e;

  // ---- the pass ----
  Stream<E> stream;
  const float slack = kSlack / c;
  float most = -kInf;  // the largest entry
  int at = -1;         // the vector that holds the first of it
  auto ask = [&](int j, int u) {
    if (j < v1 && row.is_whole(j)) copy_async(&s.ring[u][tid], row.at + (size_t)j * 16);
    copy_commit();
  };
#pragma unroll
  for (int u = 0; u < kFlight; u++) ask(v0 + tid + u * kThreads, u);
  // the first of the given tokens and, behind the pass, their logits: a chain of two loads, ahead of their use
  int token = -1;
  if (a.logp && tid < a.n) token = __ldcg(a.tokens + (size_t)row_id * a.n + tid);
  for (int j0 = v0 + tid; j0 < v1; j0 += kThreads * kFlight) {
#pragma unroll
    for (int u = 0; u < kFlight; u++) {
      const int j = j0 + u * kThreads;
      if (j >= v1) break;
      copy_wait<kFlight - 1>();
      float x[E];
      Row<BF16>::unpack(row.is_whole(j) ? s.ring[u][tid] : row.load(j), x);
      float top = fmaxf(x[0], x[1]);
#pragma unroll
      for (int i = 2; i < E; i += 2) top = max3(top, x[i], x[i + 1]);
      at = top > most ? j : at;
      most = fmaxf(most, top);
      stream.add(x, top, c, slack);
      ask(j + kFlight * kThreads, u);  // its values have been used
    }
  }
  copy_wait<0>();
  float logit = 0.f;
  if ((unsigned)token < (unsigned)a.V) logit = row.one(token);
  // ---- the CTA's sums, and each thread's largest entry ----
  // Where they are few, a thread's vectors are still in shared memory.
  const bool kept = v1 - v0 <= kFlight * kThreads;
  auto vector = [&](int j) { return kept && row.is_whole(j) ? s.ring[(j - v0) / kThreads][(j - v0) % kThreads] : row.load(j); };
  uint4 again;
  if (a.k > 0 && at >= 0) again = vector(at);
  Sums sum = stream.sums();
  auto over_warp = [&]() {
    float to = sum.b;
    for (int o = 16; o; o >>= 1) {
      to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, o));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    }
    sum.move(to, c);
    for (int o = 16; o; o >>= 1) {
      sum.s += __shfl_xor_sync(0xffffffffu, sum.s, o);
      sum.t += __shfl_xor_sync(0xffffffffu, sum.t, o);
    }
  };
  uint64_t mine = 0;
  if (a.k > 0) {
    if (at >= 0) {
      float x[E];
      Row<BF16>::unpack(again, x);
#pragma unroll
      for (int i = E - 1; i >= 0; i--)
        if (x[i] == most) mine = key_of(x[i], at * E - row.shift + i);
    }
    give_group(s, mine);
  }
  over_warp();
  if (lane == 0) s.sums[warp] = sum, s.most[warp] = most;
  if (tid == 0) s.n = s.hits = 0, s.bound = kLeast;
  __syncthreads();
  float to = s.sums[0].b;
  most = s.most[0];
#pragma unroll
  for (int w = 1; w < kWarps; w++) to = fmaxf(to, s.sums[w].b), most = fmaxf(most, s.most[w]);
  sum = Sums{to, 0.f, 0.f};
#pragma unroll
  for (int w = 0; w < kWarps; w++) {  // the same in every thread
    Sums part = s.sums[w];
    part.move(to, c);
    sum.s += part.s;
    sum.t += part.t;
  }

  // ---- its largest entries ----
  if (a.k > 0) {
    uint64_t bound = find_bound(s, a.k);
    if (a.k == 1) {  // the largest of all
      if (tid == 0) s.best[0] = bound > kLeast ? bound : 0;
      __syncthreads();
    } else {
      const int each_log2 = 32 - __clz((v1 - v0 + kThreads - 1) / kThreads - 1);  // a thread's vectors, up to a power of two
      for (;;) {
        const float least = value_of(bound);
        if (mine >= bound) s.hit[atomicAdd(&s.hits, 1)] = (uint16_t)tid;
        __syncthreads();
        const int looks = s.hits << each_log2;
        for (int w0 = tid; w0 < looks; w0 += kThreads * kLooks) {
          uint4 r[kLooks];
          int j[kLooks];
#pragma unroll
          for (int u = 0; u < kLooks; u++) {
            const int w = w0 + u * kThreads, h = w >> each_log2;
            j[u] = w < looks ? v0 + s.hit[h] + (w - (h << each_log2)) * kThreads : v1;
            if (j[u] < v1) r[u] = vector(j[u]);
          }
#pragma unroll
          for (int u = 0; u < kLooks; u++) {
            if (j[u] >= v1) continue;
            float x[E];
            Row<BF16>::unpack(r[u], x);
            float top = x[0];
#pragma unroll
            for (int i = 1; i < E; i++) top = fmaxf(top, x[i]);
            if (!(top >= least)) continue;
#pragma unroll
            for (int i = 0; i < E; i++) {
              const uint64_t key = key_of(x[i], j[u] * E - row.shift + i);
              if (key < bound || x[i] != x[i]) continue;
              const int p = atomicAdd(&s.n, 1);
              if (p < kRoom) s.found[p] = key;
            }
          }
        }
        __syncthreads();
        const int n = min(s.n, kRoom);
        const bool more = s.n > kRoom;
        __syncthreads();
        rank_found(s, n, a.k);
        if (!more) break;
        bound = s.best[a.k - 1];  // reached by k entries, and not by all that reached the last one
        __syncthreads();
        if (tid == 0) s.n = s.hits = 0;
        __syncthreads();
      }
    }
  }

  // ---- the parts of a row ----
  if (a.parts > 1) {
    static_assert(COLI_MAX_TOP <= 32, "a lane for each");
    LogprobPart* part = a.part + (size_t)row_id * a.parts;
    if (warp == 0) {  // one warp's writes: their fence is one wait
      if (lane == 0) *reinterpret_cast<float4*>(part + part_id) = make_float4(most, sum.b, sum.s, sum.t);
      if (lane < a.k) part[part_id].top[lane] = s.best[lane];
      __syncwarp();
      if (lane == 0) {
        __threadfence();
        s.last = atomicAdd(a.count + row_id, 1) == a.parts - 1;
        if (s.last) a.count[row_id] = 0;
      }
    }
    __syncthreads();
    if (!s.last) return;
    __threadfence();
    // all that the parts left is asked for at once
    constexpr int kEach = kRoom / kThreads;
    static_assert(kLogprobMostParts <= kGroups && kGroups <= kThreads, "a group for each part");
    uint64_t key[kEach], lead = 0;
    float4 left[2];
    auto of_part = [&](int p, int i) { return __ldcg(reinterpret_cast<const unsigned long long*>(&part[p].top[i])); };
#pragma unroll
    for (int h = 0; h < 2; h++) left[h] = lane + 32 * h < a.parts ? __ldcg(reinterpret_cast<const float4*>(part + lane + 32 * h)) : make_float4(-kInf, -kInf, 0.f, 0.f);
    if (a.k > 0) {
      // groups are runs of `run` of a part's keys, which descend: their first ones are their largest
      const int most_runs = kGroups / a.parts, run = (a.k + most_runs - 1) / most_runs;
      const int runs = (a.k + run - 1) / run;
      if (tid < a.parts * runs) lead = of_part(tid / runs, tid % runs * run);
#pragma unroll
      for (int u = 0; u < kEach; u++) {
        const int i = tid + u * kThreads;
        key[u] = 0;
        if (i < a.parts * a.k) key[u] = of_part(i / a.k, i % a.k);
      }
    }
    Sums two[2];
#pragma unroll
    for (int h = 0; h < 2; h++) two[h] = Sums{left[h].y, left[h].z, left[h].w};
    most = fmaxf(left[0].x, left[1].x);
    sum = two[0];
    sum.join(two[1], c);
    over_warp();
    if (a.k > 0) {
      // of the groups' largest entries the k-th largest is a bound; with fewer groups than k there is none
      if (tid < kGroups) s.group[tid] = lead;
      if (tid == 0) s.n = 0, s.bound = kLeast;
      __syncthreads();
      const uint64_t bound = find_bound(s, a.k);
#pragma unroll
      for (int u = 0; u < kEach; u++)
        if (key[u] >= bound) s.found[atomicAdd(&s.n, 1)] = key[u];
      __syncthreads();
      const int n = s.n;
      __syncthreads();
      rank_found(s, n, a.k);
    }
  }

  // ---- the answers ----
  // Of the largest entry: s is from 1 on, but for the error of what carried it there. Log p has an absolute error, a few times 2^-24: of
  // a token that is close to certain the digits of 1 - p are those that s = 1 + ... has.
  sum.move(most, c);
  const bool bad = !(sum.s < kInf);  // a NaN, or an infinity among the entries
  const bool empty = sum.s == 0.f;
  const float nan = __uint_as_float(0x7fc00000u);
  if (bad && tid == 0) set_error(a.err, COLI_E_NONFINITE);
  const float base = Sums::from(most), log_s = fmaxf(logf(sum.s), 0.f);
  auto log_p = [&](float x) {
    const float d = x - base;
    // a difference beyond binary32 of entries that are not, which the scale may bring back
    const float z = d == -kInf && x > -kInf ? fmaf(0.5f * x - 0.5f * base, 2.f * a.scale, -log_s) : fmaf(d, a.scale, -log_s);
    return bad ? nan : empty ? -kInf : z;
  };
  if (a.entropy && tid == 0) a.entropy[row_id] = bad ? nan : empty ? 0.f : fmaxf(log_s - kLn2 * (sum.t / sum.s), 0.f);
  if (a.logp)
    for (int i = tid; i < a.n; i += kThreads) {
      const size_t to = (size_t)row_id * a.n + i;
      if (i != tid) {
        token = __ldcg(a.tokens + to);
        if ((unsigned)token < (unsigned)a.V) logit = row.one(token);
      }
      if (token >= a.V) set_error(a.err, COLI_E_RANGE);
      a.logp[to] = token < 0 ? 0.f : token >= a.V ? nan : log_p(logit);
    }
  if (tid < a.k) {
    const uint64_t key = bad ? 0 : s.best[tid];
    const size_t to = (size_t)row_id * a.k + tid;
    a.top_id[to] = key ? index_of(key) : -1;
    a.top_logp[to] = key ? log_p(value_of(key)) : bad ? nan : -kInf;
  }
}

template <bool BF16>
cudaError_t launch_one(coli_ctx* ctx, const LogprobArgs& a) {
  return launch_k(logprob_kernel<BF16>, a.S * a.parts, kThreads, 0, ctx->stream, true, false, a);
}

}  // namespace

int launch_logprobs(coli_ctx* ctx, const LogprobArgs& args, int dtype) {
  LogprobArgs a = args;
  const int elem = dtype == COLI_DTYPE_BF16 ? 2 : 4, E = 16 / elem;
  a.shift_step = (int)(((uintptr_t)a.x & 15) / elem);
  const int vecs = (a.V + 2 * (E - 1)) / E;  // at most, whatever the row's shift
  a.parts = (int)(logprob_slots(ctx->num_sms) / a.S);
  a.parts = min(min(a.parts, kLogprobMostParts), (vecs + kThreads * kFew - 1) / (kThreads * kFew));
  if (a.parts < 1) a.parts = 1;
  a.per = (vecs + a.parts - 1) / a.parts;
  a.part = static_cast<LogprobPart*>(ctx->d_logprob);
  a.count = reinterpret_cast<int*>(a.part + logprob_slots(ctx->num_sms));
  a.err = ctx->d_status;
  ProfScope prof(ctx, COLI_KERNEL_LOGPROBS);
  const cudaError_t e = dtype == COLI_DTYPE_BF16 ? launch_one<true>(ctx, a) : launch_one<false>(ctx, a);
  if (e != cudaSuccess) return cuda_fail(ctx, e, "logprobs launch");
  return COLI_OK;
}

}  // namespace coli
