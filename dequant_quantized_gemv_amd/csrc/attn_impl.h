// attn_impl.h - attention of one new token per sequence over a paged
// key-value cache (gfx950).
//
// For query head h of a sequence, over the tokens t that it sees:
//   z_t = scale * q_h . K_t,   y_h = sum_t exp(z_t) V_t / sum_t exp(z_t)
// in one pass with a running maximum m: p_t = 2^(z_t log2(e) - m), and what
// was summed before is multiplied by 2^(m_old - m_new) when m rises.
//
// The matrix cores do both products.  A wave takes 32 tokens (two sub-tiles
// of 16) and up to 16 query heads that share the key-value head:
//   S^T (tokens x heads) = K Q^T,  O^T (dims x heads) += V^T P^T.
// The result of the first has in lane (g = lane / 16, j = lane % 16) head j
// and tokens 4g..4g+3 of each sub-tile, which is the second's right operand
// as it stands (the order of the summed tokens is free as long as V uses the
// same), so the probabilities never leave their registers.  V is read row by
// row, lane (g, j) taking dims j*D/16 .. of its eight tokens.  All of a lane's
// softmax state belongs to its head j.
//
// Scores: v_mfma_f32_16x16x32_f16.  fp16 keys and 8-bit codes are exact
// operands; q is split into a high and a low fp16 part (two products, about
// 22 bits), scaled by a power of two to a largest magnitude of 2^13..2^14, so
// that the parts' absolute precision is 2^-38 of the row's largest.
// Outputs: a probability may be tiny and still decide an output (where the
// likely tokens have value 0), so it keeps its 24 bits and its exponent.
// fp16 values: v_mfma_f32_16x16x4_f32, which takes p as it is.  8-bit values:
// codes are exact in bf16 and p times the value's scale is split into three
// bf16 parts, v_mfma_f32_16x16x32_bf16; the 8-bit cache has half the bytes
// per product, too few to hide the fp32 form's time.
//
// Bound by the cache's traffic where there are tokens enough: 131072 tokens of
// 8 heads x 128 in fp16 (537 MB) 101 us with the join, 5.3 TB/s; 64 sequences
// of 2048 tokens in 8 bits (277 MB) 55 us, 5.0 TB/s.  What is left there is the
// start of the workgroups and the join.  A batch of uneven lengths also waits for its longest rows: 64
// sequences of 64..4096 tokens in 8 bits (283 MB) 73 us.  One sequence of 1000
// tokens is latency: 6.5 us and 3.8 us for the join, 8.8 us together.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "attn.h"
#include "qk_common.h"
#include "qk_internal.h"

namespace qk {

typedef _Float16 h8_t __attribute__((ext_vector_type(8)));
typedef __bf16 b8_t __attribute__((ext_vector_type(8)));
typedef _Float16 h2_t __attribute__((ext_vector_type(2)));
typedef float f4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u2_t __attribute__((ext_vector_type(2)));

constexpr float kAttnLow = -3.402823466e38f;  // the running maximum before any token

// Largest / sum of the four lanes that share lane % 16, to all of them.
__device__ __forceinline__ float quad_rows_max(float v) {
    u2_t r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    v = fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
    r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    return fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}
__device__ __forceinline__ float quad_rows_sum(float v) {
    u2_t r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    v = __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
    r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}

// High and low fp16 parts of eight values (both rounded toward zero, one
// instruction for two values; the low part takes up the high part's error,
// which leaves 2^-21 of the value).
__device__ __forceinline__ void split8(const float (&p)[8], h8_t &hi, h8_t &lo) {
    u4_t h, l;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const h2_t a = __builtin_bit_cast(h2_t, __builtin_amdgcn_cvt_pkrtz(p[2 * i], p[2 * i + 1]));
        h[i] = __builtin_bit_cast(uint32_t, a);
        l[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(p[2 * i] - (float)a[0], p[2 * i + 1] - (float)a[1]));
    }
    hi = __builtin_bit_cast(h8_t, h);
    lo = __builtin_bit_cast(h8_t, l);
}

// Three bf16 parts of eight values, each the leading 8 bits of what is left:
// together all 24 bits.
__device__ __forceinline__ void split8_bf16(const float (&p)[8], b8_t (&part)[3]) {
    uint32_t r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = __builtin_bit_cast(uint32_t, p[i]);
#pragma unroll
    for (int n = 0; n < 3; ++n) {
        u4_t w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __builtin_amdgcn_perm(r[2 * i + 1], r[2 * i], 0x07060302u);
        part[n] = __builtin_bit_cast(b8_t, w);
        if (n < 2) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                r[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, r[i]) -
                                                        __builtin_bit_cast(float, r[i] & 0xFFFF0000u));
        }
    }
}

// Two bytes b, held as code + 128 in the low halves of a dword's 16-bit words
// (fp16 subnormals b * 2^-24), to fp16 code * 2^-9: exact.
__device__ __forceinline__ uint32_t codes_f16(uint32_t w) {
    const h2_t x = __builtin_bit_cast(h2_t, w);
    const h2_t c = {(_Float16)32768.0f, (_Float16)32768.0f};
    const h2_t o = {(_Float16)-0.25f, (_Float16)-0.25f};
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(x, c, o));
}

// Eight int8 codes to fp16 code * 2^-9.
__device__ __forceinline__ h8_t codes8_f16(uint32_t w0, uint32_t w1) {
    w0 ^= 0x80808080u;
    w1 ^= 0x80808080u;
    const u4_t x = {codes_f16(__builtin_amdgcn_perm(0u, w0, 0x0c010c00u)), codes_f16(__builtin_amdgcn_perm(0u, w0, 0x0c030c02u)),
                    codes_f16(__builtin_amdgcn_perm(0u, w1, 0x0c010c00u)), codes_f16(__builtin_amdgcn_perm(0u, w1, 0x0c030c02u))};
    return __builtin_bit_cast(h8_t, x);
}

template <int N> struct Bytes { uint32_t w[(N + 3) / 4]; };

template <int N>
__device__ __forceinline__ Bytes<N> load_bytes(const uint8_t *p) {
    Bytes<N> r;
    if constexpr (N % 4 != 0) r.w[N / 4] = 0;
    __builtin_memcpy(r.w, p, N);
    return r;
}

// The tokens that sequence seq of len tokens shares with its group (0 without a
// group), found by the wave's lanes; -1 where it has no result of its own to
// take part in: no tokens, fewer than are shared, or numbers above their bounds.
__device__ __forceinline__ int shared_tokens(const SharedArgs &a, int seq, int len) {
    const int lane = threadIdx.x & 63;
    int shared = 0;
    for (int g0 = 0; g0 < a.n_groups; g0 += 64) {
        const int g = min(g0 + lane, a.n_groups - 1);
        const int first = a.starts[g], end = a.starts[g + 1], n = a.shared[g];
        const uint64_t mine = __ballot(first <= seq && seq < end);
        if (mine != 0) {
            shared = max(__builtin_amdgcn_readlane(n, __builtin_ctzll(mine)), 0);
            break;
        }
    }
    const bool fine = len > 0 && len <= a.max_len && shared <= a.max_shared && len >= shared && len - shared <= a.max_own;
    return fine ? shared : -1;
}

// A workgroup's results on the way to one another: maximum and sum, outputs.
typedef float AttnWaveSums[kAttnWaves][kAttnHeads][2];
template <int D> using AttnWaveOutputs = float[kAttnWaves][kAttnHeads][D + 4];

// Workgroup `block` of `blocks`, or, where the wave takes a sequence's own tokens
// alone, four of `blocks`.
// TILED: a page holds whole sub-tiles (page_size a multiple of 16) and scales
// of neighbouring tokens lie side by side, so a sub-tile's page is looked up
// once, in scalar registers.  Otherwise lane l finds the row (and reads the
// scales) of the tile's token l % 32, and lanes take them from one another.
// With SharedArgs the tokens that a sequence has of its own, behind those that
// its group shares, always to partial results.
template <int D, bool I8, bool TILED, class ARGS>
__device__ __forceinline__ void attn_decode_block(const ARGS &a, const int block, const int blocks, AttnWaveSums &sm, AttnWaveOutputs<D> &so) {
    constexpr bool SHARED = std::is_same_v<ARGS, SharedArgs>;
    constexpr int ES = I8 ? 1 : 2;         // bytes of a key or value element
    constexpr int STEPS = D / 32;          // products over the head dimension
    constexpr int DPL = D / 16;            // dims of a lane's V row piece = tiles of O^T
    constexpr int VB = DPL * ES;           // its bytes
    constexpr int KP = I8 ? (STEPS + 1) / 2 : STEPS;  // 16-byte pieces of a lane's K row part
    typedef const __attribute__((address_space(4))) int32_t cint_t;  // scalar loads

    const int lane = threadIdx.x & 63;
    int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, j = lane & 15;
    // Chunks outermost: workgroups go round the XCDs in turn, so with chunks
    // innermost the chunks that only long sequences have would meet on the
    // same XCDs; and a sequence's first chunks, which are whole, start first.
    int b = block, waves = kAttnWaves;   // of a chunk
    if constexpr (SHARED) {
        if (a.own_waves == 1) {
            waves = 1;
            b = b * kAttnWaves + wave;
            wave = 0;
            if (b >= blocks) return;
        }
    }
    const int rows = blocks / a.nchunks;
    const int chunk = b / rows;
    b -= chunk * rows;
    const int ht = b % a.head_tiles;
    b /= a.head_tiles;
    const int kvh = b % a.n_kv;
    int seq = b / a.n_kv;
    if constexpr (SHARED) seq += a.seq0;

    const int head0 = kvh * a.group + ht * kAttnHeads;
    const int nh = min(kAttnHeads, a.group - ht * kAttnHeads);
    auto page_of = [&](int t) { return (int)((uint64_t)(uint32_t)t * a.page_magic >> a.page_shift); };

    // What waits for no other load is asked for first: the length, the first
    // tile's pages (where there is no window they follow from the chunk), q.
    const int len_in = *(cint_t *)(uintptr_t)(a.lens + seq);
    const int tbeg = chunk * a.chunk_tiles;
    int first_page[2] = {0, 0};
    if (TILED && !SHARED && a.window == 0) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int t = min(kAttnTile * (tbeg + wave) + 16 * u, a.max_len - 1);
            first_page[u] = *(cint_t *)(uintptr_t)(a.table + seq * a.ld_table + page_of(t));
        }
    }
    // lane (g, j) holds head j, the dims that its K pieces hold
    auto dim_of = [&](int s) {  // first of step s's eight dims in this lane
        if constexpr (I8) {
            if (STEPS % 2 == 1 && s == STEPS - 1) return 32 * s + 8 * g;
            return 64 * (s >> 1) + 16 * g + 8 * (s & 1);
        } else {
            return 32 * s + 8 * g;
        }
    };
    float qv[STEPS][8];
    {
        const float *q = a.q + seq * a.q_seq + (int64_t)(head0 + min(j, nh - 1)) * a.q_head;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) __builtin_memcpy(qv[s], q + dim_of(s), 32);
    }
    asm volatile("" ::: "memory");  // (keeps the loads of q ahead of those of K and V, which it does not wait for)

    const bool too_long = len_in > a.max_len;
    AttnSpan sp;
    if constexpr (SHARED) {
        const int shared = shared_tokens(a, seq, len_in);
        if (shared < 0 || len_in <= shared) return;
        sp = own_span(len_in, shared);
    } else {
        sp = attn_span(len_in < 0 ? 0 : too_long ? 0 : len_in, a.window, a.sinks);
    }
    if (!SHARED && sp.tiles == 0) {
        // no token to see: zeros (NaN where the length is past max_len)
        if (chunk == 0) {
            const float z = too_long ? __builtin_nanf("") : 0.0f;
            for (int i = threadIdx.x; i < nh * D; i += 64 * kAttnWaves) {
                const int64_t at = seq * a.y_seq + (head0 + i / D) * a.y_head + i % D;
                if (a.out_f16) static_cast<uint16_t *>(a.y)[at] = f2h(z);
                else static_cast<float *>(a.y)[at] = z;
            }
        }
        return;
    }
    const int tend = min(tbeg + a.chunk_tiles, sp.tiles);
    if (tbeg >= tend) return;  // (whole workgroup, before any barrier)

    h8_t qh[STEPS], ql[STEPS];
    int qexp = 0;
    auto split_q = [&]() __attribute__((always_inline)) {
        float top = 0.0f;
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                qv[s][i] *= a.qscale;
                top = fmaxf(top, fabsf(qv[s][i]));
            }
        top = quad_rows_max(top);
        int ex = 14;
        if (top > 0.0f && top <= 3.402823466e38f) (void)frexpf(top, &ex);
        qexp = ex - 14;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
#pragma unroll
            for (int i = 0; i < 8; ++i) qv[s][i] = ldexpf(qv[s][i], -qexp);
            split8(qv[s], qh[s], ql[s]);
        }
        if constexpr (I8) qexp += 9;  // codes are held times 2^-9
    };

    auto tile_t0 = [&](int v) { return v < sp.ns ? kAttnTile * v : sp.start + kAttnTile * (v - sp.ns); };
    // a token that is seen in the tile at t0
    auto seen_in = [&](int t0) { return t0 < a.sinks ? t0 : max(t0, sp.ws); };
    auto seen = [&](int t) { return t < sp.len && (t < a.sinks || t >= sp.ws); };

    uint32_t bad = 0;  // a page id outside the pool was met: the outputs are NaN

    auto checked = [&](int page) __attribute__((always_inline)) {
        const bool out = (unsigned)page >= (unsigned)a.n_pages;
        bad |= out ? 1u : 0u;
        return out ? 0 : page;
    };

    // Where the tile's rows are, known one tile before its loads are issued.
    // TILED: the page ids of the two sub-tiles and the slots that they begin
    // at (a sub-tile with no token that is seen takes the other's place: its
    // page may be gone).  Otherwise page and slot of the lane's token (of one
    // that is seen, if it is not).
    struct At { int page[TILED ? 2 : 1], slot[TILED ? 2 : 1]; };
    auto locate = [&](int v) __attribute__((always_inline)) {
        At at;
        const int t0 = tile_t0(v);
        if constexpr (TILED) {
            const int ts = seen_in(t0) & ~15;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                int t = t0 + 16 * u;
                if (!(t < sp.len && (t < a.sinks || t + 16 > sp.ws))) t = ts;
                const int p = page_of(t);
                at.slot[u] = t - p * a.page_size;
                at.page[u] = *(cint_t *)(uintptr_t)(a.table + seq * a.ld_table + p);
            }
        } else {
            int t = t0 + (lane & 31);
            if (!seen(t)) t = seen_in(t0);
            const int p = page_of(t);
            at.slot[0] = t - p * a.page_size;
            at.page[0] = a.table[seq * a.ld_table + p];
        }
        return at;
    };

    // sc: scales of tokens 4g + i and 16 + 4g + i, as the scores have them
    // (without TILED sc[0]: of the lane's token)
    struct Kreg { u4_t w[2][KP]; float sc[8]; } kr;
    struct Vreg { Bytes<VB> w[8]; float sc[8]; } vr;

    auto load_k_row = [&](const uint8_t *row, u4_t (&w)[KP]) __attribute__((always_inline)) {
#pragma unroll
        for (int p = 0; p < KP; ++p) {
            if constexpr (I8 && STEPS % 2 == 1) {
                if (p == KP - 1) {
                    u2_t h;
                    __builtin_memcpy(&h, row + 64 * p + 8 * g, 8);
                    w[p] = u4_t{h[0], h[1], 0, 0};
                    continue;
                }
            }
            __builtin_memcpy(&w[p], row + 64 * p + 16 * g, 16);
        }
    };
    auto row_of = [&](int page, int slot) __attribute__((always_inline)) {
        return page * a.page_stride + kvh * a.head_stride + slot * a.slot_stride;
    };
    auto scale_of = [&](int page, int slot) __attribute__((always_inline)) {
        return page * a.sc_page + kvh * a.sc_head + slot * a.sc_slot;
    };
    auto from_lane = [&](int64_t x, int src) __attribute__((always_inline)) {
        const uint32_t lo = (uint32_t)__shfl((int)(uint32_t)x, src), hi = (uint32_t)__shfl((int)(uint32_t)(x >> 32), src);
        return (int64_t)((uint64_t)hi << 32 | lo);
    };
    auto load_k = [&](const At &at) __attribute__((always_inline)) {
        if constexpr (TILED) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int page = checked(at.page[u]);
                load_k_row(a.k + row_of(page, at.slot[u]) + (uint32_t)(j * (int)a.slot_stride), kr.w[u]);
                if constexpr (I8) __builtin_memcpy(&kr.sc[4 * u], a.ks + scale_of(page, at.slot[u]) + 4 * g, 16);
            }
        } else {
            const int page = checked(at.page[0]);
            const int64_t row = row_of(page, at.slot[0]);
#pragma unroll
            for (int u = 0; u < 2; ++u) load_k_row(a.k + from_lane(row, 16 * u + j), kr.w[u]);
            if constexpr (I8) kr.sc[0] = a.ks[scale_of(page, at.slot[0])];
        }
    };
    auto load_v = [&](const At &at) __attribute__((always_inline)) {
        if constexpr (TILED) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int page = checked(at.page[u]);
                const uint8_t *base = a.v + row_of(page, at.slot[u]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    vr.w[4 * u + i] = load_bytes<VB>(base + (uint32_t)((4 * g + i) * (int)a.slot_stride + j * VB));
                if constexpr (I8) __builtin_memcpy(&vr.sc[4 * u], a.vs + scale_of(page, at.slot[u]) + 4 * g, 16);
            }
        } else {
            const int page = checked(at.page[0]);
            const int64_t row = row_of(page, at.slot[0]);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                vr.w[i] = load_bytes<VB>(a.v + from_lane(row, 16 * (i >> 2) + 4 * g + (i & 3)) + j * VB);
            if constexpr (I8) vr.sc[0] = a.vs[scale_of(page, at.slot[0])];
        }
    };
    // the scales of a lane's tokens, from the lanes that read them
    auto spread = [&](float (&sc)[8]) __attribute__((always_inline)) {
        if constexpr (I8 && !TILED) {
            const float own = sc[0];
#pragma unroll
            for (int i = 0; i < 8; ++i) sc[i] = __shfl(own, 16 * (i >> 2) + 4 * g + (i & 3));
        }
    };

    f4_t o[DPL];
#pragma unroll
    for (int c = 0; c < DPL; ++c) o[c] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
    float m = kAttnLow, l = 0.0f;

    float s[8];  // scores of tokens 4g + i (0..3) and 16 + 4g + i (4..7), in log2
    auto scores = [&]() __attribute__((always_inline)) {
        spread(kr.sc);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            f4_t c = {0.0f, 0.0f, 0.0f, 0.0f}, d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int st = 0; st < STEPS; ++st) {
                h8_t kk;
                if constexpr (I8) {
                    const u4_t &w = kr.w[u][st >> 1];
                    kk = codes8_f16(w[2 * (st & 1)], w[2 * (st & 1) + 1]);
                } else {
                    kk = __builtin_bit_cast(h8_t, kr.w[u][st]);
                }
                c = __builtin_amdgcn_mfma_f32_16x16x32_f16(kk, qh[st], c, 0, 0, 0);
                d = __builtin_amdgcn_mfma_f32_16x16x32_f16(kk, ql[st], d, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float x = c[i] + d[i];
                // a key that overflowed fp16: infinite with the high part, and
                // NaN with a low part that is 0
                if constexpr (!I8) x = __builtin_isinf(c[i]) ? c[i] : x;
                x = ldexpf(x, qexp);
                if constexpr (I8) x *= kr.sc[4 * u + i];
                s[4 * u + i] = x;
            }
        }
    };
    float p[8];  // probabilities relative to 2^m, with 8-bit values times their scales
    auto probabilities = [&](int v) __attribute__((always_inline)) {
        const int t0 = tile_t0(v);
        const bool whole = t0 + kAttnTile <= sp.len && (t0 >= sp.ws || t0 + kAttnTile <= a.sinks);
        uint32_t mask = 0xffu;
        if (!whole) {
            mask = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (seen(t0 + 16 * (i >> 2) + 4 * g + (i & 3))) mask |= 1u << i;
                else s[i] = kAttnLow;
        }
        float top = s[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) top = fmaxf(top, s[i]);
        top = quad_rows_max(top);
        if (__any(top > m)) {
            const float mn = fmaxf(m, top);
            const float f = __builtin_amdgcn_exp2f(m - mn);
            l *= f;
            m = mn;
#pragma unroll
            for (int c = 0; c < DPL; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[c][i] *= f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            p[i] = __builtin_amdgcn_exp2f(s[i] - m);
            if (!whole) p[i] = mask >> i & 1 ? p[i] : 0.0f;
            l += p[i];
        }
        if constexpr (I8) {
            spread(vr.sc);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                p[i] *= vr.sc[i];
                if (!whole) p[i] = mask >> i & 1 ? p[i] : 0.0f;
            }
        } else if (!whole) {
            // rows that are not seen may hold anything, NaN included
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int d = 0; d < (VB + 3) / 4; ++d) vr.w[i].w[d] = mask >> i & 1 ? vr.w[i].w[d] : 0u;
        }
    };
    auto outputs = [&]() __attribute__((always_inline)) {
        if constexpr (I8) {
            b8_t part[3];
            split8_bf16(p, part);
#pragma unroll
            for (int c = 0; c < DPL; ++c) {
                u4_t x;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float e0 = (float)(int8_t)(vr.w[2 * i].w[c / 4] >> (8 * (c % 4)));
                    const float e1 = (float)(int8_t)(vr.w[2 * i + 1].w[c / 4] >> (8 * (c % 4)));
                    x[i] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, e1), __builtin_bit_cast(uint32_t, e0),
                                                 0x07060302u);
                }
                const b8_t vv = __builtin_bit_cast(b8_t, x);
#pragma unroll
                for (int n = 0; n < 3; ++n) o[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vv, part[n], o[c], 0, 0, 0);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int c = 0; c < DPL; ++c) {
                    const h2_t x = __builtin_bit_cast(h2_t, vr.w[i].w[c / 2]);
                    o[c] = __builtin_amdgcn_mfma_f32_16x16x4f32((float)x[c % 2], p[i], o[c], 0, 0, 0);
                }
        }
    };

    // One register set: a tile's K registers are loaded again as soon as its
    // scores are done, its V registers as soon as its outputs are.
    int v = tbeg + wave;
    if (v < tend) {
        At at;
        if (TILED && !SHARED && a.window == 0) {
            const bool both = kAttnTile * v + 16 < sp.len;
#pragma unroll
            for (int u = 0; u < (TILED ? 2 : 1); ++u) {
                const int t = kAttnTile * v + (both ? 16 * u : 0);
                at.page[u] = both ? first_page[u] : first_page[0];
                at.slot[u] = t - page_of(t) * a.page_size;
            }
        } else {
            at = locate(v);
        }
        load_k(at);
        load_v(at);
        at = locate(min(v + waves, tend - 1));
        asm volatile("" ::: "memory");
        split_q();
        for (; v + waves < tend; v += waves) {
            const int n = v + waves;
            scores();
            load_k(at);
            probabilities(v);
            outputs();
            load_v(at);
            at = locate(min(n + waves, tend - 1));
        }
        scores();
        probabilities(v);
        outputs();
    }
    l = quad_rows_sum(l);
    if (__any(bad)) l = __builtin_nanf("");

    if constexpr (SHARED) {
        if (waves == 1) {
            if (j >= nh) return;
            float *part = a.part + ((int64_t)(seq * (int64_t)a.n_heads + head0 + j) * a.slots + a.prefix_chunks + chunk) * attn_part_floats(D);
            if (g == 0) {
                part[0] = m;
                part[1] = l;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < DPL; c += 2) {
                    const float two[2] = {o[c][i], o[c + 1][i]};
                    __builtin_memcpy(part + 4 + (4 * g + i) * DPL + c, two, 8);
                }
            return;
        }
    }

    // join the waves
    if (g == 0) {
        sm[wave][j][0] = m;
        sm[wave][j][1] = l;
    }
    if (j < nh) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < DPL; ++c) so[wave][j][(4 * g + i) * DPL + c] = o[c][i];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nh * (D / 4); i += 64 * kAttnWaves) {
        const int h = i / (D / 4), d = 4 * (i % (D / 4));
        float mm = sm[0][h][0];
#pragma unroll
        for (int w = 1; w < kAttnWaves; ++w) mm = fmaxf(mm, sm[w][h][0]);
        f4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
        float ll = 0.0f;
#pragma unroll
        for (int w = 0; w < kAttnWaves; ++w) {
            const float f = __builtin_amdgcn_exp2f(sm[w][h][0] - mm);
            ll += f * sm[w][h][1];
            const f4_t x = *reinterpret_cast<const f4_t *>(&so[w][h][d]);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] += f * x[e];
        }
        const int head = head0 + h;
        if (!SHARED && sp.tiles <= a.chunk_tiles) {
            // the only chunk
            const int64_t at = seq * a.y_seq + head * a.y_head + d;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float y = acc[e] / ll;
                if (a.out_f16) static_cast<uint16_t *>(a.y)[at + e] = f2h(y);
                else static_cast<float *>(a.y)[at + e] = y;
            }
        } else {
            int64_t slot;
            if constexpr (SHARED) slot = (int64_t)(seq * (int64_t)a.n_heads + head) * a.slots + a.prefix_chunks + chunk;
            else slot = (int64_t)(seq * (int64_t)a.n_heads + head) * a.nchunks + chunk;
            float *part = a.part + slot * attn_part_floats(D);
            if (d == 0) {
                part[0] = mm;
                part[1] = ll;
            }
            *reinterpret_cast<f4_t *>(part + 4 + d) = acc;
        }
    }
}

template <int D, bool I8, bool TILED>
__global__ __launch_bounds__(64 * kAttnWaves, D <= 128 ? 2 : 1) void attn_decode_kernel(const AttnArgs a) {
    __shared__ AttnWaveSums sm;
    __shared__ __attribute__((aligned(16))) AttnWaveOutputs<D> so;
    attn_decode_block<D, I8, TILED>(a, blockIdx.x, gridDim.x, sm, so);
}

// Joins the chunks of one (sequence, head): a workgroup's threads take the
// partial results D/4 threads at a time, kAttnJoinUnroll chunks in flight.
constexpr int kAttnJoinUnroll = 8;
template <int D>
__global__ __launch_bounds__(256) void attn_join_kernel(const AttnArgs a) {
    constexpr int COLS = D / 4;
    constexpr int ROWS = 256 / COLS;   // chunks at a time
    constexpr int U = kAttnJoinUnroll;
    __shared__ __attribute__((aligned(16))) float so[ROWS][D];
    __shared__ float sl[ROWS], sm[ROWS];
    const int head = blockIdx.x % a.n_heads;
    const int seq = blockIdx.x / a.n_heads;
    const int len_in = a.lens[seq];
    const AttnSpan sp = attn_span(len_in < 0 || len_in > a.max_len ? 0 : len_in, a.window, a.sinks);
    const int n = (sp.tiles + a.chunk_tiles - 1) / a.chunk_tiles;
    if (n <= 1) return;  // written already (whole workgroup, before any barrier)
    const float *part = a.part + (int64_t)(seq * (int64_t)a.n_heads + head) * a.nchunks * attn_part_floats(D);
    const int row = threadIdx.x / COLS, col = threadIdx.x % COLS;
    if (row < ROWS) {
        f4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
        float l = 0.0f, m = kAttnLow;
        for (int c0 = row; c0 < n; c0 += U * ROWS) {
            float pm[U], pl[U];
            f4_t x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // (past the last chunk: the last one again, with weight 0)
                const float *p = part + min(c0 + u * ROWS, n - 1) * attn_part_floats(D);
                __builtin_memcpy(&x[u], p + 4 + 4 * col, 16);
                pm[u] = p[0];
                pl[u] = p[1];
            }
            float top = m;
#pragma unroll
            for (int u = 0; u < U; ++u) top = fmaxf(top, pm[u]);
            const float f0 = __builtin_amdgcn_exp2f(m - top);
            l *= f0;
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] *= f0;
            m = top;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (c0 + u * ROWS >= n) continue;
                const float f = __builtin_amdgcn_exp2f(pm[u] - top);
                l += f * pl[u];
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[e] += f * x[u][e];
            }
        }
        *reinterpret_cast<f4_t *>(&so[row][4 * col]) = acc;
        if (col == 0) {
            sl[row] = l;
            sm[row] = m;
        }
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += 256) {
        float m = sm[0];
        for (int r = 1; r < ROWS; ++r) m = fmaxf(m, sm[r]);
        float acc = 0.0f, l = 0.0f;
        for (int r = 0; r < ROWS; ++r) {
            const float f = __builtin_amdgcn_exp2f(sm[r] - m);
            acc += f * so[r][d];
            l += f * sl[r];
        }
        const float y = acc / l;
        const int64_t at = seq * a.y_seq + head * a.y_head + d;
        if (a.out_f16) static_cast<uint16_t *>(a.y)[at] = f2h(y);
        else static_cast<float *>(a.y)[at] = y;
    }
}

template <int D, bool I8>
int attn_decode_dim(const AttnArgs &a, bool tiled, hipStream_t stream) {
    // sequences of one launch (a sequence has at most 2^20 query heads, and several
    // chunks only where all of them together have few workgroups)
    const int64_t rows = (int64_t)a.n_kv * a.head_tiles * a.nchunks;
    const int64_t most = max_groups(256) / std::max<int64_t>(rows, a.nchunks > 1 ? a.n_heads : 1);
    for (int64_t seq = 0; seq < a.n_seqs; seq += most) {
        AttnArgs p = a;
        p.n_seqs = (int)std::min<int64_t>(a.n_seqs - seq, most);
        p.q = a.q + seq * a.q_seq;
        p.y = static_cast<uint8_t *>(a.y) + seq * a.y_seq * (a.out_f16 ? 2 : 4);
        p.table = a.table + seq * a.ld_table;
        p.lens = a.lens + seq;
        if (a.part) p.part = a.part + seq * a.n_heads * a.nchunks * attn_part_floats(D);
        const dim3 grid((unsigned)(p.n_seqs * rows));
        int st = tiled ? launch(attn_decode_kernel<D, I8, true>, grid, dim3(64 * kAttnWaves), stream, p)
                       : launch(attn_decode_kernel<D, I8, false>, grid, dim3(64 * kAttnWaves), stream, p);
        if (st == QK_OK && a.nchunks > 1)
            st = launch(attn_join_kernel<D>, dim3((unsigned)(p.n_seqs * (int64_t)a.n_heads)), dim3(256), stream, p);
        if (st != QK_OK) return st;
    }
    return QK_OK;
}

template <bool I8>
int attn_decode_run(const AttnArgs &a, int head_dim, bool tiled, hipStream_t stream) {
    switch (head_dim) {
    case 32: return attn_decode_dim<32, I8>(a, tiled, stream);
    case 64: return attn_decode_dim<64, I8>(a, tiled, stream);
    case 96: return attn_decode_dim<96, I8>(a, tiled, stream);
    case 128: return attn_decode_dim<128, I8>(a, tiled, stream);
    case 160: return attn_decode_dim<160, I8>(a, tiled, stream);
    case 192: return attn_decode_dim<192, I8>(a, tiled, stream);
    case 224: return attn_decode_dim<224, I8>(a, tiled, stream);
    case 256: return attn_decode_dim<256, I8>(a, tiled, stream);
    default: return QK_ERR_INVALID_ARG;
    }
}

}  // namespace qk
