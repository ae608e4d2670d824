// Rotary positions: pairs of channels of q and k turned by position * frequency, and the table of frequencies.
//
// The angle. A frequency is a 64-bit fraction F of a turn per position, so position * F modulo 2^64 is the exact place in the
// turn: two multiplications of whole numbers, whatever the position, where binary32 would have lost the fraction from a few
// thousand turns on. Its upper 32 bits, read as a signed part of a half turn, go to sincospif.
//
// Bound by memory: q and k are read and written once. The sines and cosines of a row are shared by all of its heads, so a CTA
// takes whole rows and makes their table in shared memory while its first loads are on their way; few heads are several rows.
//
// Measured: 8191 rows of 64 + 8 heads of 128 (bf16) 53 us, 5.7 TB/s, 0.85 of a copy's rate, neighbouring channels 61 us, f32
// 90 us (0.99); 3001 f32 rows of 40 heads of 80, 36 channels turned, 18.8 us (4.1 TB/s; 22 before copies behind the turned part went two
// vectors at a time); one row 2.9 us on the device, less than the call takes on the host (7.9 us). Bound by the table's latency (plan,
// frequency, sine) at the start of each CTA. Five CTAs of 256 threads in 48 registers, which spill 12 to 20 bytes a thread, beat three
// of 384 in 56 (57 us) and four of 384 in 40 (67 us, more spills).
#include <cuda_bf16.h>

#include <cmath>
#include <type_traits>

#include "kv4.h"
#include "pipe.h"
#include "rotary.h"

namespace coli {

// f / (2 pi) * 2^64 of a frequency in radians, rounded; two doubles hold the quotient, since one would leave an error that
// 2^31 positions turn into 2^-22 of a turn.
static uint64_t turns_of(double f) {
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;  // 1 / (2 pi)
  const double hi = f * kHi;
  const double lo = std::fma(f, kHi, -hi) + f * kLo;
  const double whole = std::floor(hi);
  return (uint64_t)std::ldexp(hi - whole, 64) + (uint64_t)(int64_t)std::llrint(std::ldexp(lo, 64));
}

int rotary_freqs(int rot, double base, int scaling, double factor, double original, double low, double high, uint64_t* out) {
  if (!out || rot < 2 || rot > COLI_MAX_ROTARY_DIM || rot % 2 != 0 || !std::isfinite(base) || !(base > 1.0)) return COLI_E_INVAL;
  if (scaling < COLI_ROTARY_PLAIN || scaling > COLI_ROTARY_PARTS) return COLI_E_INVAL;
  if (scaling != COLI_ROTARY_PLAIN && (!std::isfinite(factor) || !(factor >= 1.0))) return COLI_E_INVAL;
  if (scaling == COLI_ROTARY_PARTS && (!std::isfinite(original) || !(original > 0.0) || !std::isfinite(high) || !(low >= 0.0) || !(low < high)))
    return COLI_E_INVAL;
  if (scaling == COLI_ROTARY_BASE && rot > 2) {
    base *= std::pow(factor, (double)rot / (rot - 2));
    if (!std::isfinite(base)) return COLI_E_INVAL;
  }
  for (int i = 0; i < rot / 2; i++) {
    double f = std::pow(base, -2.0 * i / rot);
    if (scaling == COLI_ROTARY_LINEAR) f /= factor;
    if (scaling == COLI_ROTARY_PARTS) {
      double g = (original * f * 0.15915494309189535 - low) / (high - low);
      g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
      f *= g + (1.0 - g) / factor;
    }
    out[i] = turns_of(f);
  }
  return COLI_OK;
}

namespace {

constexpr int kMostThreads = 256, kCtas = 5;  // CTAs of an SM; 48 registers
constexpr int kMostRows = 16;  // rows of a CTA
constexpr long long kGone = 1ll << 40, kCopied = 1ll << 41;  // not of any sequence; before its sequence's first position

// Positions of the `here` rows from row0 on, by a warp.
__device__ __forceinline__ void find_positions(const RotaryArgs& a, int row0, int here, long long* to) {
  const int lane = threadIdx.x & 31, row = row0 + lane;
  if (a.positions) {
    if (lane < here) to[lane] = __ldcg(a.positions + row);
    return;
  }
  int b = row, r0 = row, r1 = row + 1, len = 0;
  if (!a.q_start) {
    if (lane < here) len = __ldcg(a.lens + b);
  } else if (a.B < 32) {
    // the whole plan in the warp's registers: one round trip
    const int start = lane <= a.B ? __ldcg(a.q_start + lane) : 0, length = lane < a.B ? __ldcg(a.lens + lane) : 0;
    for (int l = 0; l < here; l++) {
      const unsigned le = __ballot_sync(0xffffffffu, lane < a.B && start <= row0 + l);
      const int at = max(0, __popc(le) - 1);
      const int from = __shfl_sync(0xffffffffu, start, at), until = __shfl_sync(0xffffffffu, start, at + 1);
      const int have = __shfl_sync(0xffffffffu, length, at);
      if (lane == l) r0 = from, r1 = until, len = have;
    }
  } else {
    b = kv4_seq_of(a.q_start, a.B, row0);
    if (lane < here) {
      while (b + 1 < a.B && __ldcg(a.q_start + b + 1) <= row) b++;  // a few steps: rows are neighbours
      r0 = __ldcg(a.q_start + b);
      r1 = __ldcg(a.q_start + b + 1);
      len = __ldcg(a.lens + b);
    }
  }
  if (lane >= here) return;
  // a range or a length that does not fit is reported by check_plan
  const bool owned = r0 >= 0 && r1 <= a.T && row >= r0 && row < r1;
  const long long pos = (long long)max(len, 0) - (r1 - row);
  to[lane] = !owned ? kGone : pos < 0 ? kCopied : pos;
}

// Row ranges and lengths that do not fit are reported whether or not a row falls in them.
__device__ __forceinline__ void check_plan(const RotaryArgs& a) {
  if (a.positions) return;
  for (int b = blockIdx.x * blockDim.x + threadIdx.x; b < a.B; b += gridDim.x * blockDim.x) {
    bool bad = __ldcg(a.lens + b) < 0;
    if (a.q_start) {
      const int r0 = __ldcg(a.q_start + b), r1 = __ldcg(a.q_start + b + 1);
      bad |= r0 < 0 || r1 < r0 || r1 > a.T;
    }
    if (bad) set_error(a.err, COLI_E_RANGE);
  }
}

template <int V>
struct Vec;  // V bf16 or f32 elements as they lie in memory
template <> struct Vec<16> { using T = uint4; };
template <> struct Vec<8> { using T = uint2; };
template <> struct Vec<4> { using T = uint32_t; };
template <> struct Vec<2> { using T = uint16_t; };

template <typename T>
__device__ __forceinline__ T load_cg(const void* p) {
  if constexpr (sizeof(T) == 2)
    return __ldcg(static_cast<const unsigned short*>(p));
  else if constexpr (sizeof(T) == 4)
    return __ldcg(static_cast<const unsigned int*>(p));
  else
    return __ldcg(static_cast<const T*>(p));
}

template <bool BF16, int V, typename R>
__device__ __forceinline__ void unpack(const R& raw, float (&v)[V]) {
  if constexpr (BF16 && V == 1) {
    v[0] = __uint_as_float((uint32_t)raw << 16);
  } else {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&raw);
#pragma unroll
    for (int i = 0; i < (BF16 ? V / 2 : V); i++) {
      if constexpr (BF16)
        v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      else
        v[i] = __uint_as_float(w[i]);
    }
  }
}

template <bool BF16, int V, typename R>
__device__ __forceinline__ R pack(const float (&v)[V]) {
  R raw;
  if constexpr (BF16 && V == 1) {
    raw = f32_to_bf16_rn(v[0]);
  } else {
    uint32_t* w = reinterpret_cast<uint32_t*>(&raw);
#pragma unroll
    for (int i = 0; i < (BF16 ? V / 2 : V); i++) {
      if constexpr (BF16) {
        const __nv_bfloat162 two = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&two);
      } else {
        w[i] = __float_as_uint(v[i]);
      }
    }
  }
  return raw;
}

// Positions of the CTA's rows, and the scaled cosine and sine of each pair; `my_freq` is the frequency of the thread's first
// entry of the table, asked for ahead.
__device__ __forceinline__ unsigned long long first_freq(const RotaryArgs& a, int here) {
  const int half = a.rot / 2;
  return (int)threadIdx.x < half * here ? __ldcg(reinterpret_cast<const unsigned long long*>(a.freqs) + threadIdx.x % half) : 0;
}
__device__ __forceinline__ void make_table(const RotaryArgs& a, int row0, int here, unsigned long long my_freq, long long* s_pos,
                                           float2* s_turn) {
  const int tid = threadIdx.x, half = a.rot / 2;
  if (tid < 32) find_positions(a, row0, here, s_pos);
  __syncthreads();
  for (int i = tid; i < here * half; i += blockDim.x) {
    const int r = i / half;
    const long long pos = s_pos[r];
    if (pos < kGone) {
      const unsigned long long freq = i == tid ? my_freq : __ldcg(reinterpret_cast<const unsigned long long*>(a.freqs) + (i - r * half));
      const uint32_t turn = (uint32_t)(((uint64_t)pos * freq) >> 32);
      float sine, cosine;
      sincospif((float)(int)turn * 4.656612873077393e-10f, &sine, &cosine);  // 2^-31
      s_turn[i] = make_float2(cosine * a.scale, sine * a.scale);
    }
  }
  __syncthreads();
}

__device__ __forceinline__ void rotate(float& p, float& q, float2 cs) {
  const float c = fmaf(p, cs.x, -q * cs.y), d = fmaf(q, cs.x, p * cs.y);
  p = c, q = d;
}

// i / d as a multiplication by 2^31 / d, rounded up: exact while i d < 2^31, the error being below i d.
struct Divisor {
  int d;
  uint32_t inverse;
  explicit Divisor(int d) : d(d), inverse((uint32_t)(((1ull << 31) + d - 1) / d)) {}
};
__device__ __forceinline__ int operator/(int i, const Divisor& by) { return (int)((uint64_t)i * by.inverse >> 31); }

// Tasks of a thread whose loads are under way together. Of two vectors of 8 bytes one more: 3001 f32 rows of 40 heads of 80, 36
// channels turned, 19.8 us against 21.4; a fourth spills more than it hides.
template <int BYTES>
constexpr int kTasks = BYTES <= 8 ? 3 : 2;

// Vectors of V elements. A task is two of them (two halves' worth of V pairs, or 2 V neighbouring channels); behind the turned
// part (COPY) two neighbouring ones that are copied, where there is an even number of them (`wide`), or one.
template <bool BF16, int V, bool HALF, bool COPY>
__global__ void __launch_bounds__(kMostThreads, kCtas) rotary_kernel(RotaryArgs a, int rows, bool wide, Divisor per_head, Divisor per_row) {
  constexpr int E = BF16 ? 2 : 4, U = kTasks<V * E>;
  using R = typename Vec<V * E>::T;
  extern __shared__ float2 s_turn[];  // [rows][rot / 2] cosine, sine
  __shared__ long long s_pos[kMostRows];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, threads = blockDim.x, half = a.rot / 2;
  const int row0 = blockIdx.x * rows;
  const int here = min(rows, a.T - row0);
  const int copy = wide ? 2 * V : V;  // elements of a copied vector
  const int turned = half / V, tasks = per_row.d * here;

  // A task's place: where its vectors are read and written, and which pairs they hold.
  struct Task {
    const char* in;
    char* out;
    int row, pair;  // pair < 0: a copy
  };
  auto task_of = [&](int i) {
    Task t;
    t.row = rows == 1 ? 0 : i / per_row;  // (a row alone may be longer than the division is exact for)
    i -= t.row * per_row.d;
    int head = i / per_head;
    const int v = i - head * per_head.d;
    const bool k = head >= a.side[0].heads;
    if (k) head -= a.side[0].heads;
    const RotarySide& s = a.side[k];
    const int channel = head * a.hd + (!COPY || v < turned ? (HALF ? v * V : v * 2 * V) : a.rot + (v - turned) * copy);
    t.pair = !COPY || v < turned ? v * V : -1;
    t.in = static_cast<const char*>(s.in) + ((row0 + t.row) * s.in_stride + channel) * E;
    t.out = static_cast<char*>(s.out) + ((row0 + t.row) * s.out_stride + channel) * E;
    return t;
  };
  const int apart = (HALF ? half : V) * E;  // bytes between a task's vectors

  bool made = false;
  const unsigned long long my_freq = first_freq(a, here);
  for (int first = 0; first < tasks; first += threads * U) {
    Task t[U];
    R x[U][2];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int i = first + u * threads + tid;
      t[u].row = -1;
      if (i < tasks) {
        t[u] = task_of(i);
        x[u][0] = load_cg<R>(t[u].in);
        if (!COPY || t[u].pair >= 0)
          x[u][1] = load_cg<R>(t[u].in + apart);
        else if (wide)
          x[u][1] = load_cg<R>(t[u].in + V * E);
      }
    }
    if (!made) {
      made = true;
      make_table(a, row0, here, my_freq, s_pos, s_turn);
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
      if (t[u].row < 0) continue;
      const long long pos = s_pos[t[u].row];
      if (pos == kGone) continue;
      if (pos != kCopied && (!COPY || t[u].pair >= 0)) {
        const float2* turn = s_turn + t[u].row * half + t[u].pair;
        float v[2][V];
        unpack<BF16, V>(x[u][0], v[0]);
        unpack<BF16, V>(x[u][1], v[1]);
#pragma unroll
        for (int i = 0; i < V; i++) {
          if constexpr (HALF)
            rotate(v[0][i], v[1][i], turn[i]);
          else
            rotate(v[2 * i / V][2 * i % V], v[2 * i / V][2 * i % V + 1], turn[i]);
        }
        x[u][0] = pack<BF16, V, R>(v[0]);
        x[u][1] = pack<BF16, V, R>(v[1]);
      }
      *reinterpret_cast<R*>(t[u].out) = x[u][0];
      if (!COPY || t[u].pair >= 0 || wide) *reinterpret_cast<R*>(t[u].out + (!COPY || t[u].pair >= 0 ? apart : V * E)) = x[u][1];
    }
  }
  check_plan(a);
}

// Rows whose pairs do not lie in whole vectors (an odd half, an odd stride): runs of heads pass through shared memory, read and
// written in 16-byte vectors as far as the run's own alignment goes, and are turned there element by element. A CTA takes `heads`
// heads (of q, then of k) of `rows` rows. 3001 rows of 40 heads of 80, 38 channels turned, bf16: 19 us (a
// warp for each head 25, two elements a task of the other kernel more than 30); 8191 of 72 heads of 96, 73 us (119).
template <bool BF16, bool HALF>
__global__ void __launch_bounds__(kMostThreads) rotary_run_kernel(RotaryArgs a, int rows, int heads, int runs_q, int runs, Divisor pitch, Divisor half) {
  using T = std::conditional_t<BF16, uint16_t, uint32_t>;  // an element's bits
  constexpr int E = sizeof(T);
  extern __shared__ uint4 s_raw[];  // [rows][the run, from its offset in a vector on], then the table
  __shared__ long long s_pos[kMostRows];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x;
  const int group = blockIdx.x / runs, run = blockIdx.x - group * runs;
  const int row0 = group * rows, here = min(rows, a.T - row0);
  const RotarySide& side = a.side[run >= runs_q];
  const int head0 = (run >= runs_q ? run - runs_q : run) * heads, n = min(heads, side.heads - head0);
  const int bytes = n * a.hd * E;
  float2* s_turn = reinterpret_cast<float2*>(s_raw + rows * pitch.d);
  auto at = [&](const void* p, long long stride, int r) {
    return static_cast<const char*>(p) + ((row0 + r) * stride + (long long)head0 * a.hd) * E;
  };
  const unsigned long long my_freq = first_freq(a, here);
  // vector v of row r: whole, or its elements that belong to the run
  auto each = [&](auto&& whole, auto&& element) {
    for (int i = tid; i < here * pitch.d; i += blockDim.x) {
      const int r = i / pitch, v = i - r * pitch.d, off = (int)((uintptr_t)at(side.in, side.in_stride, r) & 15);
      if (v * 16 >= off && v * 16 + 16 <= off + bytes)
        whole(r, i, v * 16 - off);
      else
#pragma unroll 1
        for (int b = max(v * 16, off); b < min(v * 16 + 16, off + bytes); b += E) element(r, i * 16 + b - v * 16, b - off);
    }
  };
  char* s_bytes = reinterpret_cast<char*>(s_raw);
  each([&](int r, int i, int b) { s_raw[i] = __ldcg(reinterpret_cast<const uint4*>(at(side.in, side.in_stride, r) + b)); },
       [&](int r, int i, int b) { *reinterpret_cast<T*>(s_bytes + i) = load_cg<T>(at(side.in, side.in_stride, r) + b); });
  make_table(a, row0, here, my_freq, s_pos, s_turn);
  for (int r = 0; r < here; r++) {
    if (s_pos[r] >= kGone) continue;
    const int off = (int)((uintptr_t)at(side.in, side.in_stride, r) & 15);
    T* row = reinterpret_cast<T*>(s_bytes + r * pitch.d * 16 + off);
    for (int w = tid; w < n * half.d; w += blockDim.x) {
      const int head = w / half, i = w - head * half.d;
      T *x = row + head * a.hd, &p = x[HALF ? i : 2 * i], &q = x[HALF ? half.d + i : 2 * i + 1];
      float u = BF16 ? bf16_to_f32((uint16_t)p) : __uint_as_float(p), v = BF16 ? bf16_to_f32((uint16_t)q) : __uint_as_float(q);
      rotate(u, v, s_turn[r * half.d + i]);
      p = BF16 ? f32_to_bf16_rn(u) : __float_as_uint(u), q = BF16 ? f32_to_bf16_rn(v) : __float_as_uint(v);
    }
  }
  __syncthreads();
  auto out = [&](int r) { return const_cast<char*>(at(side.out, side.out_stride, r)); };
  each(
      [&](int r, int i, int b) {
        if (s_pos[r] == kGone) return;
        char* to = out(r) + b;
        if (((uintptr_t)to & 15) == 0)
          *reinterpret_cast<uint4*>(to) = s_raw[i];
        else
#pragma unroll
          for (int e = 0; e < 16 / E; e++) reinterpret_cast<T*>(to)[e] = reinterpret_cast<const T*>(s_raw + i)[e];
      },
      [&](int r, int i, int b) {
        if (s_pos[r] != kGone) *reinterpret_cast<T*>(out(r) + b) = *reinterpret_cast<const T*>(s_bytes + i);
      });
  check_plan(a);
}

template <bool BF16, bool HALF>
cudaError_t launch_runs(coli_ctx* ctx, const RotaryArgs& a) {
  constexpr int E = BF16 ? 2 : 4, kBytes = 12 * 1024;  // of a CTA's runs
  const int head = a.hd * E, most = max(a.side[0].heads, a.side[1].heads);
  const int heads = max(1, min(most, kBytes / head));
  const int runs_q = (a.side[0].heads + heads - 1) / heads, runs = runs_q + (a.side[1].heads + heads - 1) / heads;
  const int rows = max(1, min(kMostRows, kBytes / (heads * head)));
  const Divisor pitch((heads * head + 15) / 16 + 1);  // of a row in shared memory, in vectors
  const size_t smem = (size_t)rows * pitch.d * 16 + (size_t)rows * (a.rot / 2) * sizeof(float2);
  // at most 12 KB of runs and two vectors a row; a table of rows * rot / 2 pairs, half of the elements at most: 24 KB
  const long long groups = (a.T + rows - 1) / rows;
  return launch_k(rotary_run_kernel<BF16, HALF>, (int)(groups * runs), kMostThreads, smem, ctx->stream, true, false, a, rows, heads, runs_q,
                  runs, pitch, Divisor(a.rot / 2));
}

template <bool BF16, int V, bool HALF>
cudaError_t launch_one(coli_ctx* ctx, const RotaryArgs& a) {
  const bool wide = (a.hd - a.rot) % (2 * V) == 0;
  const Divisor per_head(a.rot / 2 / V + (a.hd - a.rot) / (wide ? 2 * V : V)), per_row(per_head.d * (a.side[0].heads + a.side[1].heads));
  if ((long long)per_row.d * per_head.d >> 31) return launch_runs<BF16, HALF>(ctx, a);  // beyond what is divided exactly
  // whole rows, as many as keep a CTA busy, and threads that share their tasks evenly
  constexpr int U = kTasks<V * (BF16 ? 2 : 4)>;
  const int rows = max(1, min(kMostRows, 256 * U / per_row.d));
  const int rounds = (rows * per_row.d + U * kMostThreads - 1) / (U * kMostThreads);
  const int threads = ((rows * per_row.d + U * rounds - 1) / (U * rounds) + 31) / 32 * 32;
  const size_t smem = (size_t)rows * (a.rot / 2) * sizeof(float2);  // rows of 256 U tasks at most, or one: 32 KB
  return launch_k(a.hd > a.rot ? rotary_kernel<BF16, V, HALF, true> : rotary_kernel<BF16, V, HALF, false>, (a.T + rows - 1) / rows, threads, smem, ctx->stream, true, false, a, rows, wide,
                  per_head, per_row);
}

}  // namespace

int launch_rotary(coli_ctx* ctx, const RotaryArgs& args, int dtype, bool interleaved) {
  RotaryArgs a = args;
  a.err = ctx->d_status;
  const int elem = dtype == COLI_DTYPE_BF16 ? 2 : 4;
  // the widest vectors that every row, head, half and copied part is a whole number of
  long long whole = (long long)a.hd | (interleaved ? a.rot : a.rot / 2) | (a.hd - a.rot);
  uintptr_t at = 0;
  for (const RotarySide& s : a.side)
    if (s.in) {
      at |= (uintptr_t)s.in | (uintptr_t)s.out;
      if (a.T > 1) whole |= s.in_stride | s.out_stride;
    }
  if (interleaved) whole |= a.rot / 2;  // a task is two neighbouring vectors
  at |= (uintptr_t)(whole * elem);
  ProfScope prof(ctx, COLI_KERNEL_ROTARY);
  cudaError_t e;
  auto pick = [&](auto bf16, auto v16, auto v8) {
    constexpr bool kBf16 = decltype(bf16)::value;
    if (at % 16 == 0) return interleaved ? launch_one<kBf16, decltype(v16)::value, false>(ctx, a) : launch_one<kBf16, decltype(v16)::value, true>(ctx, a);
    if (at % 8 == 0) return interleaved ? launch_one<kBf16, decltype(v8)::value, false>(ctx, a) : launch_one<kBf16, decltype(v8)::value, true>(ctx, a);
    return interleaved ? launch_runs<kBf16, false>(ctx, a) : launch_runs<kBf16, true>(ctx, a);
  };
  if (dtype == COLI_DTYPE_BF16)
    e = pick(std::true_type{}, std::integral_constant<int, 8>{}, std::integral_constant<int, 4>{});
  else
    e = pick(std::false_type{}, std::integral_constant<int, 4>{}, std::integral_constant<int, 2>{});
  if (e != cudaSuccess) return cuda_fail(ctx, e, "rotary launch");
  return COLI_OK;
}

}  // namespace coli
