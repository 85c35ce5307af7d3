// gemv_x8q_n23.hip - instances of the fused quantized GEMV with stored 8-bit
// activations for 2, 3 column(s) (kernels in gemv_impl.h).
#include "gemv_impl.h"

namespace qk {

template int gemv_table_x8<2, kX8Stored>(int fmt, GemvArgs &a, bool fast, hipStream_t stream);
template int gemv_table_x8<3, kX8Stored>(int fmt, GemvArgs &a, bool fast, hipStream_t stream);

}  // namespace qk
