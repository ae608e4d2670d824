// Log probabilities: a row's log-sum-exp, entropy and largest entries in one pass over its logits.
//
// Bound by memory: every logit is read once. A CTA takes a row, or a part of one where there are few rows; the last CTA of a
// row to arrive joins the parts, in their order. A thread keeps the maximum m of what it has seen, s = sum e^(x - m) and
// t = sum (x - m) e^(x - m) (entropy = log s - t / s), and moves them when m grows.
//
// The largest entries cost the pass nothing but the place of each thread's maximum. An entry's key is its value with its index
// below, so keys never tie and the lower index wins. The maxima of 32 groups of threads are 32 entries, so the k-th largest of
// them is a bound that k entries reach at least; only threads whose own maximum reaches it look through their entries again
// (out of L2), and what they find, about k ln k entries, is ranked by comparison with one another. Where ties make it more
// than there is room for, the k-th largest of those found is a higher bound of the same kind, and the search repeats.
#include "logprobs.h"
#include "pipe.h"

namespace coli {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kRoom = kLogprobMostParts * COLI_MAX_TOP;  // entries that reach the bound
constexpr int kUnroll = 4;   // vectors of a thread in flight
constexpr float kInf = __builtin_huge_valf();
constexpr float kLowest = -3.402823466e38f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// 2^y is 0 in binary32 below this, and y 2^y then too
constexpr float kNothing = -300.f;

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

// m, s, t of a set of entries.
struct Sums {
  float m, s, t;
  // where differences are taken from: finite, so that entries of -infinity add nothing
  __device__ __forceinline__ float base() const { return fmaxf(m, kLowest); }
  // to the larger maximum `to`; c = scale log2 e
  __device__ __forceinline__ void move(float to, float c) {
    const float old = base();
    m = to;
    const float y = max_nan((old - base()) * c, kNothing), f = exp2_fast(y);
    t = f * fmaf(s, y, t);
    s *= f;
  }
  __device__ __forceinline__ void join(Sums o, float c) {
    const float to = fmaxf(m, o.m);
    move(to, c);
    o.move(to, c);
    s += o.s;
    t += o.t;
  }
};

template <bool BF16>
struct Row {
  static constexpr int E = BF16 ? 8 : 4;  // elements of a vector
  const char* at;                         // the boundary at or before the row's first element
  int shift, V;

  // vector j; elements outside the row are -infinity
  __device__ __forceinline__ uint4 load(int j) const {
    const int e0 = j * E - shift;
    const char* p = at + (size_t)j * 16;
    if (e0 >= 0 && e0 + E <= V) return __ldcg(reinterpret_cast<const uint4*>(p));
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

__device__ __forceinline__ uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }

struct Shared {
  Sums sums[kWarps];
  uint64_t group[32];
  uint64_t found[kRoom];
  uint64_t best[COLI_MAX_TOP];
  uint64_t bound;
  int n;
  bool last;
};

// The keys of s.found[0..n) that fewer than k others exceed, in order, into s.best; 0 behind them. The CTA's threads, which
// then agree.
__device__ __forceinline__ void rank_found(Shared& s, int n, int k) {
  if (threadIdx.x < COLI_MAX_TOP) s.best[threadIdx.x] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t mine = s.found[i];
    int above = 0;
    for (int j = 0; j < n; j++) above += s.found[j] > mine;
    if (above < k) s.best[above] = mine;
  }
  __syncthreads();
}

// A warp: the k-th largest of the lanes' keys (no two alike, but for 0), at least kLeast.
__device__ __forceinline__ uint64_t kth_of_warp(uint64_t key, int k) {
  int above = 0;
  for (int l = 0; l < 32; l++) above += __shfl_sync(0xffffffffu, key, l) > key;
  uint64_t at = above < k ? key : ~0ull;  // the smallest of the first k
  for (int o = 16; o; o >>= 1) {
    const uint64_t other = __shfl_xor_sync(0xffffffffu, at, o);
    at = other < at ? other : at;
  }
  return max64(at, kLeast);
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 2) logprob_kernel(LogprobArgs a) {
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
  const int v0 = part_id * a.per, v1 = min(vecs, v0 + a.per);
  const float c = a.scale * kLog2e;

  // ---- the pass ----
  Sums sum{-kInf, 0.f, 0.f};
  int at = -1;  // the vector that holds the first of the largest entries
  for (int j0 = v0 + tid; j0 < v1; j0 += kThreads * kUnroll) {
    uint4 raw[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; u++)
      if (j0 + u * kThreads < v1) raw[u] = row.load(j0 + u * kThreads);
#pragma unroll
    for (int u = 0; u < kUnroll; u++) {
      const int j = j0 + u * kThreads;
      if (j >= v1) break;
      float x[E];
      Row<BF16>::unpack(raw[u], x);
      float top = x[0];
#pragma unroll
      for (int i = 1; i < E; i++) top = fmaxf(top, x[i]);
      if (top > sum.m) {
        sum.move(top, c);
        at = j;
      }
      const float base = sum.base();
#pragma unroll
      for (int i = 0; i < E; i++) {
        const float y = max_nan((x[i] - base) * c, kNothing), e = exp2_fast(y);
        sum.s += e;
        sum.t = fmaf(e, y, sum.t);
      }
    }
  }

  // ---- the thread's largest entry, and the bound ----
  uint64_t mine = 0;
  if (a.k > 0) {
    if (at >= 0) {
      float x[E];
      Row<BF16>::unpack(row.load(at), x);
#pragma unroll
      for (int i = E - 1; i >= 0; i--)
        if (x[i] == sum.m) mine = key_of(x[i], at * E - row.shift + i);
    }
    uint64_t g = mine;
    for (int o = 8; o; o >>= 1) g = max64(g, __shfl_xor_sync(0xffffffffu, g, o));
    if ((lane & 15) == 0) s.group[tid >> 4] = g;
  }
  for (int o = 16; o; o >>= 1) {
    Sums other;
    other.m = __shfl_xor_sync(0xffffffffu, sum.m, o);
    other.s = __shfl_xor_sync(0xffffffffu, sum.s, o);
    other.t = __shfl_xor_sync(0xffffffffu, sum.t, o);
    sum.join(other, c);
  }
  if (lane == 0) s.sums[warp] = sum;
  if (tid == 0) s.n = 0;
  __syncthreads();
  sum = s.sums[0];
  for (int w = 1; w < kWarps; w++) sum.join(s.sums[w], c);  // the same in every thread
  if (a.k > 0) {
    if (warp == 0) {
      const uint64_t b = kth_of_warp(s.group[lane], a.k);
      if (lane == 0) s.bound = b;
    }
    __syncthreads();
    uint64_t bound = s.bound;
    for (;;) {
      if (mine >= bound) {
        const uint32_t least = (uint32_t)(bound >> 32);
        for (int j = v0 + tid; j < v1; j += kThreads) {
          float x[E];
          Row<BF16>::unpack(row.load(j), x);
#pragma unroll
          for (int i = 0; i < E; i++) {
            if (ordered(x[i]) < least) continue;
            const uint64_t key = key_of(x[i], j * E - row.shift + i);
            if (key < bound || x[i] != x[i]) continue;
            const int p = atomicAdd(&s.n, 1);
            if (p < kRoom) s.found[p] = key;
          }
        }
      }
      __syncthreads();
      const int n = min(s.n, kRoom);
      const bool more = s.n > kRoom;
      rank_found(s, n, a.k);
      if (!more) break;
      bound = s.best[a.k - 1];  // reached by k entries, and not by all that reached the last one
      __syncthreads();
      if (tid == 0) s.n = 0;
      __syncthreads();
    }
  }

  // ---- the parts of a row ----
  if (a.parts > 1) {
    LogprobPart* part = a.part + (size_t)row_id * a.parts;
    if (tid == 0) part[part_id].m = sum.m, part[part_id].s = sum.s, part[part_id].t = sum.t;
    if (tid < a.k) part[part_id].top[tid] = s.best[tid];
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      s.last = atomicAdd(a.count + row_id, 1) == a.parts - 1;
      if (s.last) a.count[row_id] = 0;
    }
    __syncthreads();
    if (!s.last) return;
    __threadfence();
    Sums two[2];
    for (int h = 0; h < 2; h++) {
      const int p = lane + 32 * h;
      two[h] = Sums{-kInf, 0.f, 0.f};
      if (p < a.parts) two[h] = Sums{__ldcg(&part[p].m), __ldcg(&part[p].s), __ldcg(&part[p].t)};
    }
    sum = two[0];
    sum.join(two[1], c);
    for (int o = 16; o; o >>= 1) {
      Sums other;
      other.m = __shfl_xor_sync(0xffffffffu, sum.m, o);
      other.s = __shfl_xor_sync(0xffffffffu, sum.s, o);
      other.t = __shfl_xor_sync(0xffffffffu, sum.t, o);
      sum.join(other, c);
    }
    if (a.k > 0) {
      // of the parts' largest entries the k-th largest bounds again; with fewer parts than k there is none
      auto of_part = [&](int p, int i) { return p < a.parts ? __ldcg(reinterpret_cast<const unsigned long long*>(&part[p].top[i])) : 0ull; };
      if (tid == 0) s.n = 0;
      if (warp == 0) {
        const uint64_t b = kth_of_warp(max64(of_part(lane, 0), of_part(lane + 32, 0)), a.k);
        if (lane == 0) s.bound = b;
      }
      __syncthreads();
      const uint64_t bound = s.bound;
      for (int i = tid; i < a.parts * a.k; i += kThreads) {
        const uint64_t key = of_part(i / a.k, i % a.k);
        if (key >= bound) s.found[atomicAdd(&s.n, 1)] = key;  // at most kRoom: see launch_logprobs
      }
      __syncthreads();
      rank_found(s, s.n, a.k);
    }
  }

  // ---- the answers ----
  const bool bad = !(sum.s < kInf);  // a NaN, or an infinity among the entries
  const bool empty = sum.s == 0.f;
  const float nan = __uint_as_float(0x7fc00000u);
  if (bad && tid == 0) set_error(a.err, COLI_E_NONFINITE);
  const float base = sum.base(), log_s = logf(sum.s);
  auto log_p = [&](float x) { return bad ? nan : empty ? -kInf : fmaf(x - base, a.scale, -log_s); };
  if (a.entropy && tid == 0) a.entropy[row_id] = bad ? nan : empty ? 0.f : fmaxf(log_s - kLn2 * (sum.t / sum.s), 0.f);
  if (a.logp)
    for (int i = tid; i < a.n; i += kThreads) {
      const size_t to = (size_t)row_id * a.n + i;
      const int token = __ldcg(a.tokens + to);
      if (token >= a.V) set_error(a.err, COLI_E_RANGE);
      a.logp[to] = token < 0 ? 0.f : token >= a.V ? nan : log_p(row.one(token));
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
  a.parts = min(min(a.parts, kLogprobMostParts), (vecs + kThreads - 1) / kThreads);
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
