// The binary32 instances of kv4_attn.h.
#include "kv4_attn.h"

namespace coli {

int launch_attn_f32(coli_ctx* ctx, AttnArgs& a) { return launch_shape<true>(ctx, a); }

}  // namespace coli
