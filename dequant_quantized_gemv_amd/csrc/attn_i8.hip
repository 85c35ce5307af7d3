// attn_i8.hip - instances of the paged decode attention for 8-bit caches
// (kernels in attn_impl.h).
#include "attn_impl.h"

namespace qk {

template int attn_decode_run<true>(const AttnArgs &a, int head_dim, bool tiled, hipStream_t stream);

}  // namespace qk
