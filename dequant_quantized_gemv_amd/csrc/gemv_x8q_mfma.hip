// gemv_x8q_mfma.hip - the GEMV on stored 8-bit activations for several columns,
// on the matrix cores.
//
// Per block of 32 weights the products are whole numbers,
//   I[col][row] = sum_t x_code[col][t] * w_code[row][t],
//   y[col][row] += d_w[row] * d_x[col] * I   (+ m_w[row] * (d_x[col] * sum_t x_code))
// in fp32.  One v_mfma_i32_16x16x64_i8 makes two blocks for 16 rows and 8
// columns: the left operand's rows 0..7 hold the columns' codes of the first
// block and zeros for the second, rows 8..15 the other way round.  The weights
// are the right operand, so a lane's results are weight row lane % 16 and
// four columns of one block: the weight's scale belongs to the lane, nothing
// is summed across lanes until the end, and a block costs the vector ALU about
// a dozen instructions for all columns.  The minima of four blocks times the
// scaled code sums are one v_mfma_f32_16x16x4_f32.
//
// A wave reads 16 rows x 4 blocks at a time: lane (g = lane / 16, j = lane % 16)
// the codes of block g of row j, contiguous.  Neighbouring lane groups then
// exchange halves (permlane swaps), which is all the right operand needs:
// which codes a lane has of a block does not matter as the activations are
// laid out alike.  Eight waves share 16 rows, splitting the row's blocks, and
// are summed at the end.  The window of 128 blocks that a workgroup stages is
// one pass of its waves, so all of its weights are on their way while the
// activations are staged.
//
// 11008 x 4096 at 8 columns, weights in no cache: Q4_1 12.3 us (28.2 MB; the
// kernel of gemv_impl.h, which quantizes them too, 18.7), Q4_0 11.5 (19.7), Q8_0
// 15.9 (23.7), Q5_0 12.5, Q5_1 12.7; with the weights in the Infinity Cache Q4_1
// 10.6.  That is not the weights' traffic, which a plain read moves in 5.5:
// a workgroup stages all columns (36 KB) for 16 rows (40 KB of Q4_1), so that
// half of what it moves is activations.
// Steps of four blocks per wave in flight, 1 / 2 / 4 (weights in no cache, 8
// columns): Q4_0 4096 x 4096 7.0 / 6.2 / 6.6 us, 1376 x 4096 6.8 / 5.8 / 6.2, 4096 x
// 11008 14.7 / 12.8 / 13.3; tall matrices gain a little with one step, which leaves
// room for more workgroups on a CU (Q4_1 11008 x 4096 11.3 / 12.3 / 13.1, Q4_0 32000 x
// 4096 25.3 / 25.8 / 27.8).  One block per product, whose results fill half of the
// lanes, costs 26 vector instructions a block against 12 (Q4_1 11008 x 4096 10.9
// against 10.6 us, weights in the Infinity Cache).
#include "gemv.h"
#include "qk_common.h"
#include "qk_internal.h"

#include <algorithm>
#include <type_traits>

namespace qk {

namespace {

typedef uint32_t u2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u4_t __attribute__((ext_vector_type(4)));
typedef int i4_t __attribute__((ext_vector_type(4)));
typedef float f4_t __attribute__((ext_vector_type(4)));

constexpr int kXmSteps = 2;                             // of four blocks, per wave and window
constexpr int kXmCols = 8;

template <int FMT> constexpr bool kHasMin = FMT == QK_Q4_1 || FMT == QK_Q5_1;
template <int FMT> constexpr bool kFive = FMT == QK_Q5_0 || FMT == QK_Q5_1;

template <int WINDOW> struct XmShared {
    u4_t codes[WINDOW][kXmCols][2];                     // a block's halves (x_half)
    float d[WINDOW][kXmCols];
    float ds[WINDOW][kXmCols];                          // scale times the sum of the codes
};

// The dwords that lane (g, j) reads of block g of row j: the block's own, or
// for 18-, 22- and 34-byte blocks the aligned ones that hold it (a 2-byte
// aligned 16-byte load costs half the rate: 11008 x 4096 at 8 columns, weights
// in the Infinity Cache, Q4_0 13.1 -> 9.6 us, Q8_0 19.4 -> 13.4).  Blocks begin at a dword or, every second one, in
// its middle.
template <int FMT> constexpr int kXmDwords = (Format<FMT>::kBytes + 3) / 4;

// Lane groups 1 and 3 of a against 0 and 2 of b: a becomes (a0, b0, a2, b2), b
// becomes (a1, b1, a3, b3).
__device__ __forceinline__ void swap16(uint32_t &a, uint32_t &b) {
    const u2_t r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
// Dword k (0..3) of half h of a block's 32 codes (eight dwords): as a lane
// has the weights' codes, low nibbles of eight bytes and then the high ones.
template <int FMT> __device__ __forceinline__ constexpr int x_half(int h, int k) {
    return FMT == QK_Q8_0 ? 4 * h + k : (k < 2 ? 2 * h + k : 2 + 2 * h + k);
}

// W waves per workgroup, two passes of them over a staged window.
// ALIGNED: w at a dword, an even number of blocks per row.
template <int FMT, int W, bool ALIGNED>
__global__ __launch_bounds__(64 * W) void gemv_x8q_mfma_kernel(const GemvItem it, const int nc) {
    constexpr int BS = Format<FMT>::kBytes;
    constexpr int PASS = W * kXmSteps * 4;              // blocks
    constexpr int WINDOW = 2 * PASS;
    __shared__ __attribute__((aligned(16))) XmShared<WINDOW> sh;
    __shared__ __attribute__((aligned(16))) float red[2 * W][kXmCols][16];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, j = lane & 15;
    const int row0 = 16 * blockIdx.x;
    const uint8_t *w = it.w + (int64_t)min(row0 + j, it.m - 1) * it.nb * BS;

    constexpr int ND = kXmDwords<FMT>;
    uint32_t blk[kXmSteps][ND];
    // step s of the wave's pass that begins at block `first` of the row
    auto load = [&](int first, int s) __attribute__((always_inline)) {
        // (past the row's end: its last block, which compute() leaves out)
        const int b = min(first + wave * (4 * kXmSteps) + 4 * s + g, it.nb - 1);
        const uint8_t *p = w + (int64_t)b * BS;
        if constexpr (kHasMin<FMT>) {
            __builtin_memcpy(blk[s], p, BS);
        } else if constexpr (ALIGNED) {
            // (an even block's last dword reaches into the next block of the row)
            __builtin_memcpy(blk[s], __builtin_assume_aligned(p - 2 * (b & 1), 4), 4 * ND);
        } else {
            // as an odd block lies: the scale above, then whole dwords
            uint16_t d;
            __builtin_memcpy(&d, p, 2);
            blk[s][0] = (uint32_t)d << 16;
            __builtin_memcpy(&blk[s][1], p + 2, BS - 2);
        }
    };
    // A window's activation blocks, a few per thread: their loads are issued
    // ahead of the weights' (loads complete in order), so that staging them
    // does not wait for the weights.
    constexpr int XB = WINDOW * kXmCols / (64 * W);
    uint32_t xv[XB][9];
    auto load_x = [&](int first) __attribute__((always_inline)) {
        const int n = min(WINDOW, it.nb - first);
#pragma unroll
        for (int u = 0; u < XB; ++u) {
            // (past the last block: that one again)
            const int i = min(tid + u * 64 * W, n * nc - 1);
            const int c = i / n, b = i - c * n;
            __builtin_memcpy(xv[u], it.x + c * it.ldx + (int64_t)(first + b) * (kX8BlockBytes / 4), kX8BlockBytes);
        }
        asm volatile("" ::: "memory");
    };
    auto stage = [&](int first) __attribute__((always_inline)) {
        const int n = min(WINDOW, it.nb - first);
#pragma unroll
        for (int u = 0; u < XB; ++u) {
            const int i = min(tid + u * 64 * W, n * nc - 1);
            const int c = i / n, b = i - c * n;
            int sum = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) sum = __builtin_amdgcn_sdot4((int)xv[u][1 + k], 0x01010101, sum, false);
#pragma unroll
            for (int h = 0; h < 2; ++h)
                sh.codes[b][c][h] = u4_t{xv[u][1 + x_half<FMT>(h, 0)], xv[u][1 + x_half<FMT>(h, 1)],
                                         xv[u][1 + x_half<FMT>(h, 2)], xv[u][1 + x_half<FMT>(h, 3)]};
            const float d = __builtin_bit_cast(float, xv[u][0]);
            sh.d[b][c] = d;
            if constexpr (kHasMin<FMT>) sh.ds[b][c] = d * (float)sum;
        }
    };
    f4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
    // this lane's left operand: column j % 8 of the block it is a row of
    const bool own = (j >= 8) == (g >= 2);
    // The pass at block `first` of the row, `at` of the window; a step's
    // registers are loaded with the next pass's as soon as it is done.
    auto compute = [&](int first, int at, auto more) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < kXmSteps; ++s) {
            const int b0 = at + wave * (4 * kXmSteps) + 4 * s;
            const int left = it.nb - (first + wave * (4 * kXmSteps) + 4 * s);
            if (left <= 0) break;  // (uniform; nothing is left of later passes either)
            // this lane's block: scale and minimum, fifth bits, codes
            uint32_t x[ND];
            if constexpr (kHasMin<FMT>) {
#pragma unroll
                for (int k = 0; k < ND; ++k) x[k] = blk[s][k];
            } else {
                const bool odd = !ALIGNED || (g & 1);
                x[0] = odd ? blk[s][0] >> 16 : blk[s][0];
#pragma unroll
                for (int k = 1; k < ND; ++k)
                    x[k] = odd ? blk[s][k] : __builtin_amdgcn_alignbyte(blk[s][k], blk[s][k - 1], 2);
            }
            constexpr int Q = kFive<FMT> ? 2 : 1;  // first dword of codes
            // past the row's end: weight scale 0, no activations
            if (g >= left) x[0] = 0;
            if constexpr (kHasMin<FMT>) {
                const float ds = j < 8 && g < left ? sh.ds[b0 + g][j] : 0.0f;
                acc = __builtin_amdgcn_mfma_f32_16x16x4f32(ds, h2f(x[0] >> 16), acc, 0, 0, 0);
            }
            // [p]: blocks p (lane groups 0, 1) and p + 2 (lane groups 2, 3)
            uint32_t dm[2] = {x[0], x[0]}, qh[2] = {x[1], x[1]};
            swap16(dm[0], dm[1]);
            if constexpr (kFive<FMT>) swap16(qh[0], qh[1]);
            u4_t q[2];
#pragma unroll
            for (int k = 0; k < (FMT == QK_Q8_0 ? 4 : 2); ++k) {
                uint32_t e = x[Q + k], o = x[Q + k + (FMT == QK_Q8_0 ? 4 : 2)];
                swap16(e, o);
                q[0][k] = e;
                q[1][k] = o;
            }
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int b = b0 + p + 2 * (g >> 1);   // this lane's block
                u4_t wv;
                if constexpr (FMT == QK_Q8_0) {
                    wv = q[p];
                } else {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t lo = q[p][k] & 0x0F0F0F0Fu, hi = (q[p][k] >> 4) & 0x0F0F0F0Fu;
                        if constexpr (kFive<FMT>) {
                            const uint32_t h = qh[p] >> (8 * (g & 1) + 4 * k);
                            lo |= q5_high4(h & 15u);
                            hi |= q5_high4((h >> 16) & 15u);
                        }
                        // code - 8 or - 16, byte by byte (no carries: 0x80 - offset + code < 0x100)
                        if constexpr (FMT == QK_Q4_0) {
                            lo = (lo + 0x78787878u) ^ 0x80808080u;
                            hi = (hi + 0x78787878u) ^ 0x80808080u;
                        }
                        if constexpr (FMT == QK_Q5_0) {
                            lo = (lo + 0x70707070u) ^ 0x80808080u;
                            hi = (hi + 0x70707070u) ^ 0x80808080u;
                        }
                        wv[k] = lo;
                        wv[2 + k] = hi;
                    }
                }
                const bool in = p + 2 * (g >> 1) < left;
                const u4_t xc = own && in ? sh.codes[b][j & 7][g & 1] : u4_t{0, 0, 0, 0};
                const i4_t dot = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i4_t, xc), __builtin_bit_cast(i4_t, wv),
                                                                       i4_t{0, 0, 0, 0}, 0, 0, 0);
                f4_t dx = *reinterpret_cast<const f4_t *>(&sh.d[in ? b : b0][4 * (g & 1)]);
                if (left < 4 && !in) dx = f4_t{0.0f, 0.0f, 0.0f, 0.0f};  // (an infinite scale times 0 is no 0)
                const float dw = h2f(dm[p] & 0xFFFFu);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf((float)dot[i], dw * dx[i], acc[i]);
            }
            if constexpr (decltype(more)::value) load(first + PASS, s);
        }
    };

    using T = std::true_type;
    using F = std::false_type;
    load_x(0);
#pragma unroll
    for (int s = 0; s < kXmSteps; ++s) load(0, s);
    asm volatile("" ::: "memory");
    stage(0);
    __syncthreads();
    for (int first = 0;;) {
        compute(first, 0, T{});
        compute(first + PASS, PASS, F{});
        first += WINDOW;
        if (first >= it.nb) break;
        load_x(first);
#pragma unroll
        for (int s = 0; s < kXmSteps; ++s) load(first, s);
        __syncthreads();  // readers of the previous window are done
        stage(first);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) red[2 * wave + (g >> 1)][4 * (g & 1) + i][j] = acc[i];
    __syncthreads();
    for (int i = tid; i < 16 * nc; i += 64 * W) {
        const int c = i >> 4, r = i & 15;
        float sum = red[0][c][r];
#pragma unroll
        for (int k = 1; k < 2 * W; ++k) sum += red[k][c][r];
        if (row0 + r < it.m) it.y[c * it.ldy + row0 + r] = sum;
    }
}

template <int FMT, int W, bool ALIGNED>
int start_parts(const GemvItem &it, int n, hipStream_t stream) {
    constexpr int most = (int)max_groups(64 * W) * 16;  // rows of one launch
    for (int64_t row = 0; row < it.m; row += most) {
        GemvItem p = it;
        p.w = it.w + row * it.nb * Format<FMT>::kBytes;
        p.y = it.y + row;
        p.m = (int)std::min<int64_t>(it.m - row, most);
        const dim3 grid((unsigned)((p.m + 15) / 16));
        const int st = launch(gemv_x8q_mfma_kernel<FMT, W, ALIGNED>, grid, dim3(64 * W), stream, p, n);
        if (st != QK_OK) return st;
    }
    return QK_OK;
}

template <int FMT, bool ALIGNED>
int start(const GemvItem &it, int n, hipStream_t stream) {
    // no more waves than the row's blocks need
    if (it.nb <= 8 * kXmSteps) return start_parts<FMT, 1, ALIGNED>(it, n, stream);
    if (it.nb <= 16 * kXmSteps) return start_parts<FMT, 2, ALIGNED>(it, n, stream);
    if (it.nb <= 32 * kXmSteps) return start_parts<FMT, 4, ALIGNED>(it, n, stream);
    return start_parts<FMT, 8, ALIGNED>(it, n, stream);
}

template <int FMT>
int by_alignment(const GemvItem &it, int n, hipStream_t stream) {
    if (!kHasMin<FMT> && (uintptr_t)it.w % 4 == 0 && it.nb % 2 == 0) return start<FMT, true>(it, n, stream);
    return start<FMT, false>(it, n, stream);
}

}  // namespace

int gemv_x8q_mfma(int fmt, const GemvItem &it, int n, hipStream_t stream) {
    switch (fmt) {
    case QK_Q4_0: return by_alignment<QK_Q4_0>(it, n, stream);
    case QK_Q4_1: return by_alignment<QK_Q4_1>(it, n, stream);
    case QK_Q8_0: return by_alignment<QK_Q8_0>(it, n, stream);
    case QK_Q5_0: return by_alignment<QK_Q5_0>(it, n, stream);
    case QK_Q5_1: return by_alignment<QK_Q5_1>(it, n, stream);
    default: return QK_ERR_INVALID_ARG;
    }
}

}  // namespace qk
