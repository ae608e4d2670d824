// Attention over the 4-bit key/value cache: the choice of the kernel, and the bf16 instances of kv4_attn.h.
#include "kv4_attn.h"

namespace coli {

// Query rows per sequence and key/value head, on average, from which the tensor-core tiles of kv4_tile.cu take over: up
// to 16 rows one pass of kv4_attn.h serves them all; from 17 on it reads and unpacks the cache again for every 16. Eight
// requests with 30 rows each: up to 300 tokens 20 us there and 21 us with tiles, 1000 tokens 27 and 27, 3000 tokens 40 and
// 38, 20011 tokens 113 and 87; 8192 rows over 10007 tokens 4.9 ms and 0.46 ms. The average hides a mix: a prompt chunk of
// 512 rows among 64 decoding requests of 4000 tokens takes the tiles for all of them, 357 us where the two kinds called
// apart take 81 and 79. Tiles are made for bf16 and heads of at most 128 channels (tensor memory holds two 128-row outputs).
constexpr int kTileFrom = 17;

int launch_attn_bf16(coli_ctx* ctx, AttnArgs& a) { return launch_shape<false>(ctx, a); }

int launch_kv4_attention(coli_ctx* ctx, const Kv4View& c, const Kv4Plan& p, const void* q, long long q_stride, int dtype,
                         int q_heads, float scale, int window, void* out, long long out_stride) {
  const bool f32 = dtype == COLI_DTYPE_F32;
  if (!f32 && c.hd <= 128 && (long long)p.T * (q_heads / c.heads) >= (long long)kTileFrom * p.B)
    return launch_kv4_tiles(ctx, c, p, q, q_stride, q_heads, scale, window, out, out_stride);
  const size_t elem = f32 ? 4 : 2;
  AttnArgs a{c, p, q, q_stride, q_heads / c.heads, scale, window, out, out_stride};
  a.vec = ((uintptr_t)q % 16 == 0) && (q_stride * elem) % 16 == 0;
  a.vec_out = ((uintptr_t)out % (4 * elem) == 0) && out_stride % 4 == 0;
  a.count = ctx->d_kv_count;
  a.err = ctx->d_status;
  a.wait_ns = ctx->wait_ns ? ctx->wait_ns : kWaitLimitNs;
  a.withhold = ctx->test_withhold > 0;
  if (a.withhold) ctx->test_withhold--;
  return f32 ? launch_attn_f32(ctx, a) : launch_attn_bf16(ctx, a);
}

}  // namespace coli
