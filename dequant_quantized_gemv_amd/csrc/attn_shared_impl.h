// attn_shared_impl.h - attention of one new token per sequence where groups of
// sequences share their first tokens (gfx950): those are read once per group.
//
// Two launches.  In the first, some workgroups take the shared tokens for all
// query rows of a group (every sequence's heads that share a key-value head: a
// matrix product instead of a product per row) and others each sequence's own
// tokens as the decode kernel does; both leave partial results (running maximum,
// sum and output) that the join combines.
//
// Shared tokens: a workgroup of four waves takes a tile of query rows over one
// chunk of the shared tokens.  Keys and values go through LDS in tiles, keys
// as they are and values transposed, so that both products read their operands
// 16 bytes at a time, and v_mfma_f32_32x32x16 takes 32 rows per wave:
//   S^T (tokens x rows) = K Q^T,  O^T (dims x rows) += V^T P^T.
// Of a result tile lane (g = lane / 32, j = lane % 32) has row j and tokens
// 8 (r / 4) + 4 g + r % 4; the second product's right operand wants eight tokens of
// one g in a lane, and since their order is free as long as both operands have
// the same, the values' tokens are stored in the order that the results have.
// The next tile's rows are in registers while one is worked on.
// A workgroup has 128 rows, every wave all tokens of a tile, or, where groups
// have no more, 64 or 32, two or four waves taking parts of a tile's tokens for the
// same rows, joined in LDS at the end: fewer partial results per row, and no
// waves without rows (8 rows of 32768 tokens of head size 128 44.3 / 45.8 us with
// 64 / 128, 64 rows 114 / 102; 32 rows take tiles of 128 tokens, which registers hold up
// to head size 64: 32 groups of 16 rows there 28.2 -> 25.5, at 128 spilled, 44 -> 59).
//
// Scores as in the decode kernel: exact keys, q in two fp16 parts.  The low
// part is never 0 beside a high part that is not (fp16's least value is added to
// it, 2^-37 of the row's largest), so that a key which overflowed to infinity
// keeps its sign.  Probabilities: with 8-bit values
// all 24 bits in three bf16 parts; with fp16 values two fp16 parts of 2^12 p,
// which holds p within 2^-21 of itself and 2^-36 of the row's largest (the exact form,
// v_mfma_f32_16x16x4_f32, has an eighth of the rate, and this kernel is bound
// by its products).
//
// What bounds it: long shared parts their products (64 sequences of 4 x 8 heads of 128 over
// 32768 tokens: 101 us, of which 66 grow with the tokens: 1.05 PFLOP/s with the second
// parts; the rest is beginnings and ends, own tokens and the join), few rows the
// traffic (8 sequences: 43 us, of which 22 grow with the tokens, 6.1 TB/s), own tokens
// what bounds the decode kernel, before and not beside the rest: from head size 96 up (and
// with 64 or more rows at 64) the registers leave room for two workgroups to a CU, below
// that for three.  Own tokens go first; shared ones first, or
// one after the other in turn, took 64 x 32768 from 104 to 120 us.  8 bits spend more
// vector instructions than products (12 to a product against 6 in fp16, to make fp16
// keys, bf16 values and three parts of the probabilities); at head size 128 4 (64 rows) to
// 7 (128) registers are spilled, outside the loop.  Above 128 q's parts and
// the outputs fill the 256 vector registers, and the loop moves others to and from the
// accumulation registers (at 256 2.6 moves to a product; 64 sequences of 2 x 8 heads of 256
// over 16384 tokens 71 us where their products are 31).
// Groups are found by looking through all of them, 64 at a time, in every workgroup: up to
// 64 it is one step, 1024 groups of 2 sequences behind 512 tokens take 776 us where the decode
// kernel takes 645, 4096 sequences of groups of their own 1540 against 219.
#pragma once

#include "attn_impl.h"

namespace qk {

typedef float f16_t __attribute__((ext_vector_type(16)));

template <int D>
struct PrefixLds {
    static constexpr int BN = prefix_tokens(D);
    static constexpr int kRow = 2 * D + 16;    // bytes of a key row (the 16 keep 16-byte reads of 16 rows off each other's banks)
    static constexpr int kDim = 2 * BN + 16;   // bytes of a dimension's values
    static constexpr int kValues = BN * kRow;
    static constexpr int kPlaces = kValues + D * kDim;     // places of the next two tiles' rows
    static constexpr int kScales = kPlaces + 2 * BN * 8;   // scales of the tile's keys, then values
    static constexpr int kBytes = kScales + 2 * BN * 4;
};

// Sum and largest of the two lanes that share lane % 32.
__device__ __forceinline__ float pair_max(float v) {
    const u2_t r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    return fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}
__device__ __forceinline__ float pair_sum(float v) {
    const u2_t r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}

// High and low fp16 parts of eight values: the high one rounded toward zero, the
// low one the rounded difference (one mixed-precision fma makes it; minus is -1,
// held where the compiler does not know it and make a subtraction of it).
__device__ __forceinline__ void split8_mixed(const float (&p)[8], float minus, h8_t &hi, h8_t &lo) {
    u4_t h;
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(p[2 * i], p[2 * i + 1]));
    hi = __builtin_bit_cast(h8_t, h);
#pragma unroll
    for (int i = 0; i < 8; ++i) lo[i] = (_Float16)__builtin_fmaf((float)hi[i], minus, p[i]);
}

template <int D, bool I8, int WM>
__device__ __forceinline__ void attn_prefix_block(const SharedArgs &a, const int block, uint8_t *lds) {
    constexpr int ROWS = prefix_rows(WM), BN = prefix_tokens(D);
    constexpr int WN = 4 / WM;                 // waves that take different tokens of the same rows
    constexpr int SUBS = BN / WN / 32;         // 32-token blocks of a wave
    constexpr int ES = I8 ? 1 : 2;
    constexpr int KS = D / 16, DB = D / 32;    // steps of the first product; blocks of output dims
    constexpr int NQ = BN / 4;                 // quads of tokens
    constexpr int UNITS = NQ * (D / 8);        // four tokens by eight dims each
    constexpr int NU = (UNITS + 255) / 256;    // of a thread
    using L = PrefixLds<D>;
    int64_t *places = reinterpret_cast<int64_t *>(lds + L::kPlaces);
    float *scales = reinterpret_cast<float *>(lds + L::kScales);

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 5, j = lane & 31;
    const int wn = wave / WM, row0 = 32 * (wave % WM);

    // The row tiles of one chunk and head are neighbours on one XCD, whose L2
    // then has the chunk's rows for all of them but the first.  How many row tiles
    // there are is known here only: workgroups without one come last (among the
    // others they left CUs with half of their work: 148 -> 121 us for 64 x 32768).
    const int units = a.n_kv * a.prefix_chunks;
    int at = 0, n = 0, sh = 0, tiles = 0, upto = 0;   // a lane's group, 64 groups at a time
    auto groups_from = [&](int g0) __attribute__((always_inline)) {
        const int gi = g0 + lane;
        at = n = sh = 0;
        if (gi < a.n_groups) {
            at = min(max(a.starts[gi], 0), a.n_seqs);
            n = (min(max(a.starts[gi + 1], at), a.n_seqs) - at) * a.group;
            sh = a.shared[gi];
        }
        upto = tiles = (n + ROWS - 1) / ROWS;
        // (sums of the lanes up to each: within rows of 16, then over the rows)
        upto += __builtin_amdgcn_update_dpp(0, upto, 0x111, 0xF, 0xF, false);   // row_shr:1
        upto += __builtin_amdgcn_update_dpp(0, upto, 0x112, 0xF, 0xF, false);
        upto += __builtin_amdgcn_update_dpp(0, upto, 0x114, 0xF, 0xF, false);
        upto += __builtin_amdgcn_update_dpp(0, upto, 0x118, 0xF, 0xF, false);
        upto += __builtin_amdgcn_update_dpp(0, upto, 0x142, 0xA, 0xF, false);   // row_bcast:15
        upto += __builtin_amdgcn_update_dpp(0, upto, 0x143, 0xC, 0xF, false);   // row_bcast:31
    };
    int total = 0;
    for (int g0 = 0; g0 < a.n_groups; g0 += 64) {
        groups_from(g0);
        total += __builtin_amdgcn_readlane(upto, 63);
    }
    // (groups out of order may add up to anything; their rows are NaN in the end)
    if (total <= 0 || total > a.row_tiles) return;
    const int nth = (block >> 3) + a.group0;
    const int unit = nth / total * 8 + (block & 7);
    if (unit >= units) return;
    const int kvh = unit % a.n_kv, chunk = unit / a.n_kv;
    int tile = nth % total;

    // the group that the row tile is of
    int first = 0, rows = 0, shared = 0;
    for (int g0 = 0; g0 < a.n_groups; g0 += 64) {
        if (a.n_groups > 64) groups_from(g0);
        const uint64_t past = __ballot(upto > tile);
        if (past != 0) {
            const int src = __builtin_ctzll(past);
            first = __builtin_amdgcn_readlane(at, src);
            rows = __builtin_amdgcn_readlane(n, src);
            shared = __builtin_amdgcn_readlane(sh, src);
            tile -= __builtin_amdgcn_readlane(upto, src) - __builtin_amdgcn_readlane(tiles, src);
            break;
        }
        tile -= __builtin_amdgcn_readlane(upto, 63);
    }
    if (tile < 0 || (int64_t)tile * ROWS >= rows) return;
    if (shared <= 0 || shared > a.max_shared) return;
    const int64_t chunk_tokens = (int64_t)a.prefix_tiles * BN;
    if (chunk * chunk_tokens >= shared) return;
    const int t0 = (int)(chunk * chunk_tokens);
    const int t1 = (int)min((int64_t)shared, t0 + chunk_tokens);
    const int ntiles = (t1 - t0 + BN - 1) / BN;
    const int wrow = tile * ROWS + row0;               // the wave's first row
    const int left = rows - wrow;                      // of its 32
    const int row = wrow + min(j, max(left, 1) - 1);   // lane's (one that is there)
    const int member = row / a.group;
    const int members = rows / a.group;
    const int seq = first + min(member, members - 1);
    const int head = kvh * a.group + row - member * a.group;

    // places of the rows of a tile's tokens, one thread each; past the end
    // the last token's again
    const int32_t *table = a.table + first * a.ld_table;
    const int first_len = *(const __attribute__((address_space(4))) int32_t *)(uintptr_t)(a.lens + first);
    uint32_t bad = 0;
    auto token_of = [&](int n) { return (int)min((int64_t)t0 + (int64_t)n * BN + tid, (int64_t)t1 - 1); };
    auto page_of = [&](int t) { return (int)((uint64_t)(uint32_t)t * a.page_magic >> a.page_shift); };
    float sc0[2] = {0.0f, 0.0f}, sc1[2] = {0.0f, 0.0f};   // scales of this tile's token and of the next one's
    auto place = [&](int n, int id, float (&sc)[2]) __attribute__((always_inline)) {
        const bool out = (unsigned)id >= (unsigned)a.n_pages;
        bad |= out ? 1u : 0u;
        const int t = token_of(n), page = out ? 0 : id;
        const int slot = t - page_of(t) * a.page_size;
        places[(n & 1) * BN + tid] = page * a.page_stride + kvh * a.head_stride + slot * a.slot_stride;
        if constexpr (I8) {
            const int64_t at = page * a.sc_page + kvh * a.sc_head + slot * a.sc_slot;
            sc[0] = a.ks[at];
            sc[1] = a.vs[at];
        }
    };

    // A first sequence that was dropped or cut short has ids outside the pool where
    // its pages were: a chunk with such a page is read by the row of the first
    // sequence that has all shared tokens (there is none: nobody has a result).
    auto living = [&]() __attribute__((always_inline)) {
        bool gone = false;
        for (int p = page_of(t0) + lane; p <= page_of(t1 - 1); p += 64) gone = gone || (unsigned)table[p] >= (unsigned)a.n_pages;
        if (!__any(gone)) return first;
        for (int s = 0; s < members; s += 64) {
            const uint64_t has = __ballot(s + lane < members && a.lens[first + min(s + lane, members - 1)] >= shared);
            if (has != 0) return __builtin_amdgcn_readfirstlane(first + s + __builtin_ctzll(has));
        }
        return first;
    };

    struct Quad { uint32_t k[4][2 * ES], v[4][2 * ES]; } reg[NU];
    // Pieces of a row that neighbouring lanes read: eight where they divide it, whole
    // lines of 128 bytes in fp16 (16 groups of 8 rows, head size 64, 60 us with four, 60 with
    // eight that meet on the same banks in LDS, 52 with eight; 8 bits gain nothing).
    constexpr int PIECES = std::min((D / 8) & -(D / 8), 8);
    auto unit_at = [&](int u, int &quad, int &piece) {
        quad = (u / PIECES) % NQ;
        piece = PIECES * (u / PIECES / NQ) + u % PIECES;
    };
    // Where a dimension has the tokens at `pos` (every 16 dimensions in another
    // order: eight neighbouring pieces would be stored to the same banks).
    auto swizzled = [&](int dim, int pos) { return pos ^ (16 * (dim >> 4 & 3)); };
    auto load = [&](int n) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < NU; ++i) {
            const int u = tid + 256 * i;
            if (UNITS % 256 != 0 && u >= UNITS) continue;
            int quad, piece;
            unit_at(u, quad, piece);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t at = places[(n & 1) * BN + 4 * quad + e] + 8 * ES * piece;
                __builtin_memcpy(reg[i].k[e], a.k + at, 8 * ES);
                __builtin_memcpy(reg[i].v[e], a.v + at, 8 * ES);
            }
        }
    };
    auto store = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < NU; ++i) {
            const int u = tid + 256 * i;
            if (UNITS % 256 != 0 && u >= UNITS) continue;
            int quad, piece;
            unit_at(u, quad, piece);
            const int pos = 16 * (quad >> 2) + 8 * (quad & 1) + 2 * (quad & 2);  // of the quad's tokens in the results' order
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                h8_t kk;
                if constexpr (I8) kk = codes8_f16(reg[i].k[e][0], reg[i].k[e][1]);
                else __builtin_memcpy(&kk, reg[i].k[e], 16);
                *reinterpret_cast<h8_t *>(lds + (4 * quad + e) * L::kRow + 16 * piece) = kk;
            }
#pragma unroll
            for (int d = 0; d < 8; ++d) {
                u2_t w;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if constexpr (I8) {
                        const float e0 = (float)(int8_t)(reg[i].v[2 * h][d / 4] >> (8 * (d % 4)));
                        const float e1 = (float)(int8_t)(reg[i].v[2 * h + 1][d / 4] >> (8 * (d % 4)));
                        w[h] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, e1), __builtin_bit_cast(uint32_t, e0), 0x07060302u);
                    } else {
                        w[h] = __builtin_amdgcn_perm(reg[i].v[2 * h + 1][d / 2], reg[i].v[2 * h][d / 2],
                                                     d % 2 ? 0x07060302u : 0x05040100u);
                    }
                }
                *reinterpret_cast<u2_t *>(lds + L::kValues + (8 * piece + d) * L::kDim + 2 * swizzled(8 * piece, pos)) = w;
            }
        }
    };

    // q is asked for first, and then the places of the first rows
    float qv[KS][8];
    {
        const float *q = a.q + seq * a.q_seq + head * a.q_head + 8 * g;
#pragma unroll
        for (int s = 0; s < KS; ++s) __builtin_memcpy(qv[s], q + 16 * s, 32);
    }
    asm volatile("" ::: "memory");
    int p0 = 0, p1 = 0, id = 0;
    auto first_pages = [&]() __attribute__((always_inline)) {
        if (tid < BN) {
            p0 = table[page_of(token_of(0))];
            p1 = table[page_of(token_of(1))];
            id = table[page_of(token_of(2))];
        }
    };
    first_pages();
    if (first_len < shared) {   // (asked for beside the length that tells whether the row has them)
        table = a.table + living() * a.ld_table;
        first_pages();
    }
    if (tid < BN) {
        place(0, p0, sc0);
        place(1, p1, sc1);
    }
    __syncthreads();
    load(0);

    // q in two parts
    h8_t qh[KS], ql[KS];
    int qexp;
    {
        float top = 0.0f;
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                qv[s][i] *= a.qscale;
                top = fmaxf(top, fabsf(qv[s][i]));
            }
        top = pair_max(top);
        int ex = 14;
        if (top > 0.0f && top <= 3.402823466e38f) (void)frexpf(top, &ex);
        qexp = ex - 14;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
#pragma unroll
            for (int i = 0; i < 8; ++i) qv[s][i] = ldexpf(qv[s][i], -qexp);
            split8(qv[s], qh[s], ql[s]);
            if constexpr (!I8) {
                // (fp16's least value with the high part's sign is added where that is not 0:
                // 2^-37 of the row's largest; the low part has the same sign or is 0)
                typedef uint16_t s8_t __attribute__((ext_vector_type(8)));
                const s8_t h = __builtin_bit_cast(s8_t, qh[s]);
                const s8_t some = __builtin_elementwise_min((s8_t)(h & (uint16_t)0x7FFF), (s8_t)(uint16_t)1);
                ql[s] += __builtin_bit_cast(h8_t, (s8_t)(some | (h & (uint16_t)0x8000)));
            }
        }
        if constexpr (I8) qexp += 9;  // codes are held times 2^-9
    }
    // (where 2^qexp is no normal number, all scores are 0 to the last bit either way)
    const float back = ldexpf(1.0f, max(qexp, -126));

    // Probabilities are held times 2^LIFT, and the maximum that they are relative
    // to follows the largest score only where that is past it by SLACK (2^15 is what
    // fp16 has room for): rows of one wave seldom rise together.
    constexpr float LIFT = I8 ? 0.0f : 12.0f, SLACK = 3.0f;
    f16_t o[DB];
#pragma unroll
    for (int c = 0; c < DB; ++c)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[c][r] = 0.0f;
    float m = kAttnLow, l = 0.0f;               // m: the running maximum less LIFT
    float minus = -1.0f;
    asm("" : "+s"(minus));

    for (int n = 0; n < ntiles; ++n) {
        __syncthreads();   // (the last tile and its places are read)
        store();
        if (tid < BN) {
            if constexpr (I8) {
                scales[tid] = sc0[0];
                scales[BN + tid] = sc0[1];
                sc0[0] = sc1[0];
                sc0[1] = sc1[1];
            }
            place(n + 2, id, sc1);
        }
        __syncthreads();
        if (tid < BN) id = table[page_of(token_of(n + 3))];
        if (n + 1 < ntiles) load(n + 1);
        if (left <= 0) continue;
#pragma unroll
        for (int sub = 0; sub < SUBS; ++sub) {
            const int b0 = (SUBS * wn + sub) * 32;   // the block's first token in the tile
            const int here = t1 - t0 - n * BN - b0;  // tokens from there on
            if (here <= 0) continue;
            // all operands of a product are asked for before its first instruction
            h8_t kk[KS];
#pragma unroll
            for (int s = 0; s < KS; ++s) kk[s] = *reinterpret_cast<const h8_t *>(lds + (b0 + j) * L::kRow + 32 * s + 16 * g);
            __builtin_amdgcn_sched_barrier(0);
            f16_t c;
#pragma unroll
            for (int r = 0; r < 16; ++r) c[r] = 0.0f;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                c = __builtin_amdgcn_mfma_f32_32x32x16_f16(kk[s], qh[s], c, 0, 0, 0);
                c = __builtin_amdgcn_mfma_f32_32x32x16_f16(kk[s], ql[s], c, 0, 0, 0);
            }
            u4_t vv[2][DB];
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int c2 = 0; c2 < DB; ++c2)
                    vv[s][c2] = *reinterpret_cast<const u4_t *>(lds + L::kValues + (32 * c2 + j) * L::kDim + 2 * swizzled(32 * c2 + j, b0 + 16 * s + 8 * g));
            __builtin_amdgcn_sched_barrier(0);
            float p[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                p[r] = c[r];
                if constexpr (I8) p[r] *= scales[b0 + 8 * (r >> 2) + 4 * g + (r & 3)];
            }
            if (here < 32) {
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (8 * (r >> 2) + 4 * g + (r & 3) >= here) p[r] = -__builtin_inff();
            }
            float top = p[0];
#pragma unroll
            for (int r = 1; r < 16; ++r) top = __builtin_elementwise_maximum(top, p[r]);
            top = __builtin_fmaf(pair_max(top), back, -LIFT);
            if (__any(top > m + SLACK)) {
                const float mn = fmaxf(m, top);
                const float f = __builtin_amdgcn_exp2f(m - mn);
                l *= f;
                m = mn;
#pragma unroll
                for (int c2 = 0; c2 < DB; ++c2)
#pragma unroll
                    for (int r = 0; r < 16; ++r) o[c2][r] *= f;
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                p[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(p[r], back, -m));
                l += p[r];
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                float ps[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) ps[i] = p[8 * s + i];
                if constexpr (I8) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        ps[i] *= scales[BN + b0 + 16 * s + 8 * (i >> 2) + 4 * g + (i & 3)];
                        // (the scale of a token past the end is the last one's: 0 where that is not finite)
                        if (here < 32 && 16 * s + 8 * (i >> 2) + 4 * g + (i & 3) >= here) ps[i] = 0.0f;
                    }
                    b8_t part[3];
                    split8_bf16(ps, part);
#pragma unroll
                    for (int c2 = 0; c2 < DB; ++c2) {
                        const b8_t w = __builtin_bit_cast(b8_t, vv[s][c2]);
#pragma unroll
                        for (int e = 0; e < 3; ++e) o[c2] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w, part[e], o[c2], 0, 0, 0);
                    }
                } else {
                    h8_t hi, lo;
                    split8_mixed(ps, minus, hi, lo);
#pragma unroll
                    for (int c2 = 0; c2 < DB; ++c2) {
                        const h8_t w = __builtin_bit_cast(h8_t, vv[s][c2]);
                        o[c2] = __builtin_amdgcn_mfma_f32_32x32x16_f16(w, hi, o[c2], 0, 0, 0);
                        o[c2] = __builtin_amdgcn_mfma_f32_32x32x16_f16(w, lo, o[c2], 0, 0, 0);
                    }
                }
            }
        }
    }
    l = pair_sum(l);
    if (__syncthreads_or(bad)) l = __builtin_nanf("");

    if constexpr (WN > 1) {
        // the results of waves with the same rows, the first one's registers taking them all
        float *other = reinterpret_cast<float *>(lds);
        constexpr int PER = (16 * DB + 2) * 64;
        static_assert(4 * PER * (4 - WM) <= L::kPlaces, "waves' results in the tile's place");
        if (wn > 0) {
            float *mine = other + (wave - WM) * PER;
#pragma unroll
            for (int c = 0; c < DB; ++c)
#pragma unroll
                for (int r = 0; r < 16; ++r) mine[(16 * c + r) * 64 + lane] = o[c][r];
            mine[16 * DB * 64 + lane] = m;
            mine[(16 * DB + 1) * 64 + lane] = l;
        }
        __syncthreads();
        if (wn > 0) return;
        float ms[WN], mm = m;
#pragma unroll
        for (int w = 1; w < WN; ++w) {
            ms[w] = other[((w - 1) * WM + wave) * PER + 16 * DB * 64 + lane];
            mm = fmaxf(mm, ms[w]);
        }
        const float f0 = __builtin_amdgcn_exp2f(m - mm);
        l *= f0;
#pragma unroll
        for (int c = 0; c < DB; ++c)
#pragma unroll
            for (int r = 0; r < 16; ++r) o[c][r] *= f0;
#pragma unroll
        for (int w = 1; w < WN; ++w) {
            const float f = __builtin_amdgcn_exp2f(ms[w] - mm);
            const float *from = other + ((w - 1) * WM + wave) * PER + lane;
            l += f * from[(16 * DB + 1) * 64];
#pragma unroll
            for (int c = 0; c < DB; ++c)
#pragma unroll
                for (int r = 0; r < 16; ++r) o[c][r] += f * from[(16 * c + r) * 64];
        }
        m = mm;
    }
    if (j >= left) return;
    float *part = a.part + ((int64_t)(seq * (int64_t)a.n_heads + head) * a.slots + chunk) * attn_part_floats(D);
    if (g == 0) {
        part[0] = m;
        part[1] = l;
    }
#pragma unroll
    for (int c = 0; c < DB; ++c)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            *reinterpret_cast<f4_t *>(part + 4 + 32 * c + 8 * r + 4 * g) =
                f4_t{o[c][4 * r], o[c][4 * r + 1], o[c][4 * r + 2], o[c][4 * r + 3]};
}

// One launch for both: own tokens (bound by memory, of uneven lengths) first,
// so that the shared ones fill the CUs as those end.
template <int D, bool I8, bool TILED, int WM>
__global__ __launch_bounds__(256, D <= 128 ? 2 : 1) void attn_shared_kernel(const SharedArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    if ((int)blockIdx.x < a.own_blocks) {
        auto &sm = *reinterpret_cast<AttnWaveSums *>(lds);
        auto &so = *reinterpret_cast<AttnWaveOutputs<D> *>(lds + sizeof(AttnWaveSums));
        attn_decode_block<D, I8, TILED>(a, blockIdx.x, a.own_items, sm, so);
    } else {
        // (a multiple of 8 behind the own tokens' workgroups, for the XCDs)
        const int block = (int)blockIdx.x - (a.own_blocks + 7) / 8 * 8;
        if (block >= 0) attn_prefix_block<D, I8, WM>(a, block, lds);
    }
}

// Joins the partial results of one (sequence, head): those of the shared
// tokens' chunks, then those of its own.
template <int D, int T>
__global__ __launch_bounds__(T) void attn_shared_join_kernel(const SharedArgs a) {
    constexpr int COLS = D / 4;
    constexpr int ROWS = T / COLS;     // chunks at a time
    constexpr int U = kAttnJoinUnroll;
    __shared__ __attribute__((aligned(16))) float so[ROWS][D];
    __shared__ float sl[ROWS], sm[ROWS];
    const int head = blockIdx.x % a.n_heads;
    const int seq = blockIdx.x / a.n_heads + a.seq0;
    const int len = a.lens[seq];
    const int shared = shared_tokens(a, seq, len);
    // groups out of order have no result
    bool order = true;
    for (int g = threadIdx.x & 63; g < a.n_groups; g += 64) {
        const int first = a.starts[g], end = a.starts[g + 1];
        order = order && first >= 0 && first <= end && end <= a.n_seqs;
    }
    const bool in_order = __all(order);
    const bool fine = in_order && shared >= 0;
    const int row = threadIdx.x / COLS, col = threadIdx.x % COLS;
    int n1 = 0, n = 0;
    if (fine) {
        const int64_t chunk = (int64_t)a.prefix_tiles * prefix_tokens(D);
        n1 = shared > 0 ? (int)((shared + chunk - 1) / chunk) : 0;
        n = n1 + (len > shared ? (own_span(len, shared).tiles + a.chunk_tiles - 1) / a.chunk_tiles : 0);
    }
    const float *part = a.part + (int64_t)(seq * (int64_t)a.n_heads + head) * a.slots * attn_part_floats(D);
    if (row < ROWS && n > 0) {
        f4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
        float l = 0.0f, m = kAttnLow;
        for (int c0 = row; c0 < n; c0 += U * ROWS) {
            float pm[U], pl[U];
            f4_t x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // (past the last chunk: the last one again, with weight 0)
                const int c = min(c0 + u * ROWS, n - 1);
                const float *p = part + (c < n1 ? c : a.prefix_chunks + c - n1) * attn_part_floats(D);
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
    for (int d = threadIdx.x; d < D; d += T) {
        float y = __builtin_nanf("");
        if (n > 0) {
            float m = sm[0];
            for (int r = 1; r < ROWS; ++r) m = fmaxf(m, sm[r]);
            float acc = 0.0f, l = 0.0f;
            for (int r = 0; r < ROWS; ++r) {
                const float f = __builtin_amdgcn_exp2f(sm[r] - m);
                acc += f * so[r][d];
                l += f * sl[r];
            }
            y = acc / l;
        } else if (len <= 0 && in_order) {
            y = 0.0f;
        }
        const int64_t at = seq * a.y_seq + head * a.y_head + d;
        if (a.out_f16) static_cast<uint16_t *>(a.y)[at] = f2h(y);
        else static_cast<float *>(a.y)[at] = y;
    }
}

template <int D, bool I8, bool TILED, int WM>
int attn_shared_start(const SharedArgs &a, hipStream_t stream) {
    constexpr size_t bytes = std::max<size_t>(PrefixLds<D>::kBytes, sizeof(AttnWaveSums) + sizeof(AttnWaveOutputs<D>));
    const auto kern = attn_shared_kernel<D, I8, TILED, WM>;
    if (bytes > 65536 && hipFuncSetAttribute(reinterpret_cast<const void *>(kern), hipFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)bytes) != hipSuccess)
        return QK_ERR_LAUNCH;
    // workgroups of the shared tokens in eights, one for each XCD, and of a sequence's own
    const int64_t eights = a.prefix_chunks > 0 ? ((int64_t)a.n_kv * a.prefix_chunks + 7) / 8 * a.row_tiles : 0;
    const int64_t each = (int64_t)a.n_kv * a.head_tiles * a.nchunks, most = max_groups(256) / 8 * 8;
    const int64_t items = kAttnWaves / a.own_waves;   // of a workgroup
    auto go = [&](int64_t seq, int64_t n, int64_t eight, int64_t ne) {
        SharedArgs p = a;
        p.seq0 = (int)seq;
        p.own_items = (int)(n * each);
        p.own_blocks = (int)((n * each + items - 1) / items);
        p.group0 = (int)eight;
        return launch_lds(kern, dim3((unsigned)((p.own_blocks + 7) / 8 * 8 + 8 * ne)), dim3(256), bytes, stream, p);
    };
    if (a.n_seqs * each <= most - 8 * eights) return go(0, a.n_seqs, 0, eights);
    int st = QK_OK;
    for (int64_t i = 0; i < eights && st == QK_OK; i += most / 8) st = go(0, 0, i, std::min(eights - i, most / 8));
    for (int64_t i = 0; i < a.n_seqs && st == QK_OK; i += most / each) st = go(i, std::min<int64_t>(a.n_seqs - i, most / each), 0, 0);
    return st;
}

template <int D, bool I8, int WM>
int attn_shared_tiled(const SharedArgs &a, bool tiled, hipStream_t stream) {
    return tiled ? attn_shared_start<D, I8, true, WM>(a, stream) : attn_shared_start<D, I8, false, WM>(a, stream);
}

template <int D, bool I8>
int attn_shared_dim(const SharedArgs &a, bool tiled, hipStream_t stream) {
    int st;
    if (a.row_waves == 4) st = attn_shared_tiled<D, I8, 4>(a, tiled, stream);
    else if (a.row_waves == 2) st = attn_shared_tiled<D, I8, 2>(a, tiled, stream);
    else if constexpr (prefix_tokens(D) == 128) st = attn_shared_tiled<D, I8, 1>(a, tiled, stream);
    else return QK_ERR_INVALID_ARG;
    // A wave joins a row of few partial results where there are many rows, four
    // waves otherwise (8192 rows of 9 23 / 16 us with four / one, 2048 rows of 33 10 / 11;
    // the whole call with 2048 rows of 17 66.6 / 68.3).
    const bool one_wave = a.slots <= 16 && (int64_t)a.n_seqs * a.n_heads >= 1024;
    const int64_t most = max_groups(256) / a.n_heads;  // sequences of one launch
    for (int64_t i = 0; i < a.n_seqs && st == QK_OK; i += most) {
        SharedArgs p = a;
        p.seq0 = (int)i;
        const dim3 grid((unsigned)(std::min<int64_t>(a.n_seqs - i, most) * a.n_heads));
        st = one_wave ? launch(attn_shared_join_kernel<D, 64>, grid, dim3(64), stream, p)
                      : launch(attn_shared_join_kernel<D, 256>, grid, dim3(256), stream, p);
    }
    return st;
}

template <bool I8>
int attn_shared_run(const SharedArgs &a, int head_dim, bool tiled, hipStream_t stream) {
    switch (head_dim) {
    case 32: return attn_shared_dim<32, I8>(a, tiled, stream);
    case 64: return attn_shared_dim<64, I8>(a, tiled, stream);
    case 96: return attn_shared_dim<96, I8>(a, tiled, stream);
    case 128: return attn_shared_dim<128, I8>(a, tiled, stream);
    case 160: return attn_shared_dim<160, I8>(a, tiled, stream);
    case 192: return attn_shared_dim<192, I8>(a, tiled, stream);
    case 224: return attn_shared_dim<224, I8>(a, tiled, stream);
    case 256: return attn_shared_dim<256, I8>(a, tiled, stream);
    default: return QK_ERR_INVALID_ARG;
    }
}

}  // namespace qk
