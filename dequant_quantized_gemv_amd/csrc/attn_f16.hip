// attn_f16.hip - instances of the paged decode attention for fp16 caches
// (kernels in attn_impl.h).
#include "attn_impl.h"

namespace qk {

template int attn_decode_run<false>(const AttnArgs &a, int head_dim, bool tiled, hipStream_t stream);

}  // namespace qk
