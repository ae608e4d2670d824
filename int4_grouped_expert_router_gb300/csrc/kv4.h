// The 4-bit key/value cache: its layout in memory, the plan of a batch, and the launchers of the
// calls on it (kv4.cu: write and read back; kv4_attn.cu: attention).
//
// Layout. The cache is a row of units of 16 tokens of one head, a page's units of one head next to
// each other: unit (page, head, token / 16) starts at
//   ((page * heads + head) * (page_tokens / 16) + token / 16) * kv4_unit_bytes.
// So whatever the page size, any run of tokens of a page and head is one contiguous block that a
// single bulk copy can fetch, codes and scales together. A unit holds, in order:
//   key codes    8 hd bytes, key scales   [16 tokens][ng] (scale | offset << 16, two bf16)
//   value codes  8 hd bytes, value scales [16 tokens][ng]
// The codes lie as the matrix instructions' A fragments want them, so that a warp's lane reads all
// of its codes of a unit with consecutive 16-byte loads (lane = 4 r + c, r < 8, c < 4; iw = min(hd/32, 4)
// words of 8 codes per load, the word index i = channel / 32 counting first within iw):
//   keys (A = K, rows are tokens): word i of token t, quarter c holds channels 32 i + 8 c + 0..7 in
//     its nibbles 0..7. A group of gs >= 32 channels is a run of whole words i.
//   values (A = V^T, rows are channels): word i of token pair p = t / 2, row r holds in its low half
//     token 2p and in its high half token 2p + 1, nibble j the channel 32 i + 16 (j / 2) + 2 r + j % 2.
//     A lane thus reads two neighbouring tokens of a channel as the two halves of one register, which
//     is what the instruction multiplies along the token axis.
// A token's part of a value word is 16 bits of its own, so tokens are written without touching the
// other half.
#pragma once

#include "coli_internal.h"

namespace coli {

constexpr int kKvUnit = 16;  // tokens of a unit
constexpr long long kKvMaxLen = (1ll << 31) - 256;  // longest sequence: positions rounded up to a stage stay below 2^31

__host__ __device__ constexpr uint32_t kv4_unit_bytes(int hd, int ng) { return (uint32_t)(16 * hd + 128 * ng); }
// Offsets of a unit's parts.
__host__ __device__ constexpr uint32_t kv4_kscale_at(int hd) { return (uint32_t)(8 * hd); }
__host__ __device__ constexpr uint32_t kv4_v_at(int hd, int ng) { return (uint32_t)(8 * hd + 64 * ng); }
__host__ __device__ constexpr uint32_t kv4_vscale_at(int hd, int ng) { return (uint32_t)(16 * hd + 64 * ng); }

// Byte offset within the key codes of the word of token t (0..15), channels 32 i + 8 c + 0..7.
__host__ __device__ constexpr uint32_t kv4_k_word(int hd, int t, int i, int c) {
  const int iw = hd / 32 < 4 ? hd / 32 : 4;
  return (uint32_t)((i / iw) * 256 * iw + t * 16 * iw + c * 4 * iw + (i % iw) * 4);
}
// Byte offset within the value codes of the word of token pair p (0..7), row r, word i.
__host__ __device__ constexpr uint32_t kv4_v_word(int hd, int p, int r, int i) {
  const int iw = hd / 32 < 4 ? hd / 32 : 4;
  return (uint32_t)((p / 4) * 4 * hd + (i / iw) * 128 * iw + (r * 4 + p % 4) * 4 * iw + (i % iw) * 4);
}

struct Kv4View {
  uint8_t* base;
  int pages, heads, page_log2, hd, ng;
};

// A batch: see the header. T rows, B sequences.
struct Kv4Plan {
  const int32_t* q_start;
  const int32_t* lens;
  const int32_t* table;
  int T, B, table_stride;
};

int launch_kv4_append(coli_ctx* ctx, const Kv4View& c, const Kv4Plan& p, const void* k, long long k_stride, const void* v,
                      long long v_stride, int dtype);
int launch_kv4_read(coli_ctx* ctx, const Kv4View& c, const Kv4Plan& p, void* k, long long k_stride, void* v,
                    long long v_stride, int dtype);
int launch_kv4_attention(coli_ctx* ctx, const Kv4View& c, const Kv4Plan& p, const void* q, long long q_stride, int dtype,
                         int q_heads, float scale, int window, void* out, long long out_stride);

// The tensor-core form for many query rows per sequence (kv4_tile.cu): bf16, hd 64 or 128.
int launch_kv4_tiles(coli_ctx* ctx, const Kv4View& c, const Kv4Plan& p, const void* q, long long q_stride, int q_heads,
                     float scale, int window, void* out, long long out_stride);

#ifdef __CUDACC__

__device__ __forceinline__ const uint8_t* kv4_unit(const Kv4View& c, int page, int head, int off) {
  const size_t unit = ((size_t)page * c.heads + head) * (size_t)(1 << (c.page_log2 - 4)) + (off >> 4);
  return c.base + unit * kv4_unit_bytes(c.hd, c.ng);
}

// Whether a group's scale | offset << 16 is of values that are not finite: NaN, or an offset that has rounded to infinity.
__device__ __forceinline__ bool kv4_broken(uint32_t par) { return (par & 0x7f800000u) == 0x7f800000u; }

// The rows [r0, r1) of sequence b, made safe: an order or a range that does not fit gives an empty range
// and the error.
__device__ __forceinline__ void kv4_rows(const Kv4Plan& p, int b, int& r0, int& r1, int* err) {
  if (!p.q_start) {
    r0 = b;
    r1 = b + 1;
    return;
  }
  r0 = __ldcg(p.q_start + b);
  r1 = __ldcg(p.q_start + b + 1);
  if (r0 < 0 || r1 < r0 || r1 > p.T) {
    set_error(err, COLI_E_RANGE);
    r0 = r1 = 0;
  }
}

// The last sequence b with q_start[b] <= row, found by a whole warp, 32 entries at a time. Whatever q_start (not NULL) holds,
// the result is a sequence of 0..B-1; the caller checks that it owns the row.
__device__ __forceinline__ int kv4_seq_of(const int32_t* q_start, int B, int row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, at < hi && __ldcg(q_start + at) <= row);
    lo += max(0, __popc(le) - 1) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// The first position that a row at position pos sees (pos may be negative: such a row sees nothing). Any window goes: no
// difference is formed that could pass 32 bits.
__device__ __forceinline__ int kv4_from(int pos, int window) { return window > 0 && pos >= window ? pos - window + 1 : 0; }

// The most tokens that a sequence can have.
__device__ __forceinline__ long long kv4_most(const Kv4Plan& p, int page_log2) {
  return min((long long)p.table_stride << page_log2, kKvMaxLen);
}

// The length of sequence b, clamped to what its table can name.
__device__ __forceinline__ int kv4_len(const Kv4Plan& p, int page_log2, int b, int* err) {
  const int len = __ldcg(p.lens + b);
  const long long most = kv4_most(p, page_log2);
  if (len < 0 || len > most) {
    set_error(err, COLI_E_RANGE);
    return len < 0 ? 0 : (int)most;
  }
  return len;
}

#endif

}  // namespace coli
