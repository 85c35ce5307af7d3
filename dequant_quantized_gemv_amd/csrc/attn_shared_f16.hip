// attn_shared_f16.hip - instances of the attention with shared first tokens for
// fp16 caches (kernels in attn_shared_impl.h).
#include "attn_shared_impl.h"

namespace qk {

template int attn_shared_run<false>(const SharedArgs &a, int head_dim, bool tiled, hipStream_t stream);

}  // namespace qk
