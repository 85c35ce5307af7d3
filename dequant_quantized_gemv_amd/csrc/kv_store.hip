// kv_store.hip - new keys and values into a paged cache, rounded to fp16 or
// quantized to 8 bits with one scale per token and head.
//
// A group of 8..64 lanes takes one row (head_dim elements of one token and
// head, key or value), four elements per lane, so a row is read once and the
// 8-bit scale's maximum is a few lane exchanges.  Bound by the traffic of
// the rows; at decode sizes by the launch.
#include "attn.h"
#include "qk_common.h"
#include "qk_internal.h"

namespace qk {

namespace {

typedef float f4_t __attribute__((ext_vector_type(4)));

template <int GS, bool I8>
__global__ __launch_bounds__(256) void kv_store_kernel(const StoreArgs a) {
    const int64_t row = ((int64_t)blockIdx.x * 256 + threadIdx.x) / GS;
    const int e = 4 * (threadIdx.x % GS);
    if (row >= 2 * a.rows) return;  // (whole groups)
    const int kind = row >= a.rows;
    const int r = (int)(kind ? row - a.rows : row);
    const int tok = r / a.n_kv, head = r - tok * a.n_kv;
    // a row that has no place in the cache is left out
    const int seq = a.seq ? a.seq[tok] : tok;
    const int pos = a.pos[tok];
    if ((unsigned)seq >= (unsigned)a.n_seqs || pos < 0) return;
    const int p = pos / a.page_size;
    if (p >= a.max_pages) return;
    const int page = a.table[seq * a.ld_table + p];
    if ((unsigned)page >= (unsigned)a.n_pages) return;
    const int slot = pos - p * a.page_size;
    const bool in = e < a.head_dim;
    const float *src = kind ? a.v + tok * a.v_tok + head * a.v_head : a.k + tok * a.k_tok + head * a.k_head;
    f4_t x = {0.0f, 0.0f, 0.0f, 0.0f};
    if (in) __builtin_memcpy(&x, src + e, 16);
    const int64_t at = page * a.page_stride + head * a.head_stride + slot * a.slot_stride + e;
    uint8_t *dst = kind ? a.vc : a.kc;
    if constexpr (I8) {
        // d = max|x| / 127, codes x / d rounded half to even (both divisions
        // rounded as IEEE has them); a row with an infinite or NaN value has
        // d = NaN and codes 0
        float top = 0.0f;
        bool fine = true;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            top = fmaxf(top, fabsf(x[i]));
            fine = fine && fabsf(x[i]) <= 3.402823466e38f;
        }
        if (!fine) top = __builtin_inff();
#pragma unroll
        for (int d = 1; d < GS; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
        const float d = top <= 3.402823466e38f ? top / 127.0f : __builtin_nanf("");
        uint32_t q = 0;
        if (d > 0.0f) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // (the bound holds but for a subnormal d, which may be well below max|x| / 127)
                const float c = fminf(fmaxf(rintf(x[i] / d), -127.0f), 127.0f);
                q |= ((uint32_t)(int)c & 0xFFu) << (8 * i);
            }
        }
        if (in) *reinterpret_cast<uint32_t *>(dst + at) = q;
        if (e == 0) (kind ? a.vs : a.ks)[page * a.sc_page + head * a.sc_head + slot * a.sc_slot] = d;
    } else if (in) {
        uint2 h;
        h.x = (uint32_t)f2h(x[0]) | ((uint32_t)f2h(x[1]) << 16);
        h.y = (uint32_t)f2h(x[2]) | ((uint32_t)f2h(x[3]) << 16);
        *reinterpret_cast<uint2 *>(dst + 2 * at) = h;
    }
}

template <bool I8>
int run(const StoreArgs &a, hipStream_t stream) {
    const int gs = a.head_dim <= 32 ? 8 : a.head_dim <= 64 ? 16 : a.head_dim <= 128 ? 32 : 64;
    const dim3 grid((unsigned)((2 * a.rows * gs + 255) / 256));
    switch (gs) {
    case 8: return launch(kv_store_kernel<8, I8>, grid, dim3(256), stream, a);
    case 16: return launch(kv_store_kernel<16, I8>, grid, dim3(256), stream, a);
    case 32: return launch(kv_store_kernel<32, I8>, grid, dim3(256), stream, a);
    default: return launch(kv_store_kernel<64, I8>, grid, dim3(256), stream, a);
    }
}

}  // namespace

int launch_kv_store(const StoreArgs &a, bool i8, hipStream_t stream) {
    return i8 ? run<true>(a, stream) : run<false>(a, stream);
}

}  // namespace qk
