// kv_store.hip - new keys and values into a paged cache, rounded to fp16 or
// quantized to 8 bits with one scale per token and head.
//
// A group of 8..64 lanes takes one token and head, key and value row (head_dim
// elements), four elements of each per lane: a row is read once, the 8-bit
// scale's maximum is a few lane exchanges, and one lookup serves both rows.
// Bound by the traffic of the rows, at decode sizes by the launch and the
// chain of lookups: 64 tokens of 8 x 128 take 2.5 us to fp16 and 3.3 to 8 bits,
// 4000 take 10.6 (49 MB, 5.4 TB/s past the launch) and 12.9 to 8 bits (41 MB).  Eight elements
// per lane: 2.5, 10.4 and 11.8, and 6.8 against 6.5 for 1500 tokens to 8 bits;
// two tokens per group 12.7, key and value rows in groups of their own 13.5.
#include <algorithm>

#include "attn.h"
#include "qk_common.h"
#include "qk_internal.h"

namespace qk {

namespace {

typedef float f4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u2_t __attribute__((ext_vector_type(2)));

constexpr int kStoreLane = 4;  // elements per lane

// A row's elements, held by GS neighbouring lanes, to int8 codes and the row's
// scale: d = max|x| / 127, codes x / d rounded half to even (both divisions
// rounded as IEEE has them); a row with an infinite or NaN value has d = NaN
// and codes 0.
template <int GS>
__device__ __forceinline__ uint32_t row_codes(const float (&x)[kStoreLane], float &d) {
    float top = 0.0f;
    bool fine = true;
#pragma unroll
    for (int i = 0; i < kStoreLane; ++i) {
        top = fmaxf(top, fabsf(x[i]));
        fine = fine && fabsf(x[i]) <= 3.402823466e38f;
    }
    if (!fine) top = __builtin_inff();
    top = fmaxf(top, dpp<0xB1>(top));                                 // quad_perm [1,0,3,2]
    top = fmaxf(top, dpp<0x4E>(top));                                 // quad_perm [2,3,0,1]
    top = fmaxf(top, dpp<0x141>(top));                                // row_half_mirror: 8 lanes
    if constexpr (GS >= 16) top = fmaxf(top, dpp<0x140>(top));        // row_mirror: 16 lanes
    if constexpr (GS >= 32) top = fmaxf(top, __shfl_xor(top, 16));
    if constexpr (GS >= 64) top = fmaxf(top, __shfl_xor(top, 32));
    d = top <= 3.402823466e38f ? top / 127.0f : __builtin_nanf("");
    if (!(d > 0.0f)) return 0;
    // A product with the reciprocal is within 127 * 2^-22 of the quotient, so
    // unless it lies that near a tie both round to the same whole number; the
    // division proper (ten instructions a value) is left to lanes where it
    // does, or where the reciprocal of a subnormal d overflows.
    const float r = __builtin_amdgcn_rcpf(d);
    float c[kStoreLane];
    bool sure = true;
#pragma unroll
    for (int i = 0; i < kStoreLane; ++i) {
        const float y = x[i] * r;
        c[i] = rintf(y);
        sure = sure && fabsf(y - c[i]) <= 0.4999f;
    }
    if (!sure) {
#pragma unroll
        for (int i = 0; i < kStoreLane; ++i) c[i] = rintf(x[i] / d);
    }
    uint32_t q = 0;
#pragma unroll
    for (int i = 0; i < kStoreLane; ++i) {
        // (the bound holds but for a subnormal d, which may be well below max|x| / 127)
        q |= ((uint32_t)(int)fminf(fmaxf(c[i], -127.0f), 127.0f) & 0xFFu) << (8 * i);
    }
    return q;
}

template <int GS, bool I8>
__global__ __launch_bounds__(256) void kv_store_kernel(const StoreArgs a) {
    // A workgroup takes neighbouring tokens of one head, whose places are
    // neighbours too when the tokens are a prompt's.
    constexpr int R = 256 / GS;
    const int64_t block = blockIdx.x / a.n_kv;
    const int head = blockIdx.x - (int)block * a.n_kv;
    const int64_t tok = block * R + threadIdx.x / GS;
    const int e = kStoreLane * (threadIdx.x % GS);
    if (tok >= a.tokens) return;  // (whole groups)
    const bool in = e < a.head_dim;
    // the rows do not wait for their place in the cache
    float x[2][kStoreLane] = {};
    if (in) {
        __builtin_memcpy(x[0], a.k + tok * a.k_tok + head * a.k_head + e, sizeof(x[0]));
        __builtin_memcpy(x[1], a.v + tok * a.v_tok + head * a.v_head + e, sizeof(x[1]));
    }
    asm volatile("" ::: "memory");
    // a row that has no place in the cache is left out
    const int seq = a.seq ? a.seq[tok] : (int)tok;
    const int pos = a.pos[tok];
    if ((unsigned)seq >= (unsigned)a.n_seqs || pos < 0) return;
    const int p = pos / a.page_size;
    if (p >= a.max_pages) return;
    const int page = a.table[seq * a.ld_table + p];
    if ((unsigned)page >= (unsigned)a.n_pages) return;
    const int slot = pos - p * a.page_size;
    const int64_t at = page * a.page_stride + head * a.head_stride + slot * a.slot_stride + e;
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
        uint8_t *dst = kind ? a.vc : a.kc;
        const auto &v = x[kind];
        if constexpr (I8) {
            float d;
            const uint32_t q = row_codes<GS>(v, d);
            if (in) *reinterpret_cast<uint32_t *>(dst + at) = q;
            if (e == 0) (kind ? a.vs : a.ks)[page * a.sc_page + head * a.sc_head + slot * a.sc_slot] = d;
        } else if (in) {
            u2_t h;
#pragma unroll
            for (int i = 0; i < 2; ++i) h[i] = (uint32_t)f2h(v[2 * i]) | ((uint32_t)f2h(v[2 * i + 1]) << 16);
            *reinterpret_cast<u2_t *>(dst + 2 * at) = h;
        }
    }
}

template <int GS, bool I8>
int start(const StoreArgs &a, hipStream_t stream) {
    constexpr int R = 256 / GS;
    const int64_t most = max_groups(256) / a.n_kv * R;  // tokens of one launch
    for (int64_t tok = 0; tok < a.tokens; tok += most) {
        StoreArgs p = a;
        p.tokens = std::min(a.tokens - tok, most);
        p.k = a.k + tok * a.k_tok;
        p.v = a.v + tok * a.v_tok;
        p.pos = a.pos + tok;
        if (a.seq) {
            p.seq = a.seq + tok;
        } else {
            // (token i is of sequence i)
            p.n_seqs = (int)std::max<int64_t>(a.n_seqs - tok, 0);
            p.table = a.table + (p.n_seqs > 0 ? tok * a.ld_table : 0);
        }
        const dim3 grid((unsigned)((p.tokens + R - 1) / R * a.n_kv));
        const int st = launch(kv_store_kernel<GS, I8>, grid, dim3(256), stream, p);
        if (st != QK_OK) return st;
    }
    return QK_OK;
}

template <bool I8>
int run(const StoreArgs &a, hipStream_t stream) {
    if (a.head_dim <= 32) return start<8, I8>(a, stream);
    if (a.head_dim <= 64) return start<16, I8>(a, stream);
    if (a.head_dim <= 128) return start<32, I8>(a, stream);
    return start<64, I8>(a, stream);
}

}  // namespace

int launch_kv_store(const StoreArgs &a, bool i8, hipStream_t stream) {
    return i8 ? run<true>(a, stream) : run<false>(a, stream);
}

}  // namespace qk
