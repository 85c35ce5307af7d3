// attn_shared_i8.hip - instances of the attention with shared first tokens for
// 8-bit caches (kernels in attn_shared_impl.h).
#include "attn_shared_impl.h"

namespace qk {

template int attn_shared_run<true>(const SharedArgs &a, int head_dim, bool tiled, hipStream_t stream);

}  // namespace qk
