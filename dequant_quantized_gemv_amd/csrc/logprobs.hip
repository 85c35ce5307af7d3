// logprobs.hip - log probabilities of given tokens, entropy and the best
// alternatives of rows of logits.
//
// With M the row's largest logit, z_i = scale * (x_i - M), S = sum exp(z_i):
//   log p_i = z_i - ln S,   H = ln S - sum exp(z_i) z_i / S.
// A part of a row is read once and stays in the registers of a workgroup,
// which takes M, then S and the weighted sum, then the best from there.  The
// logits equal to M are counted and not summed, so that ln S = log1p(S - 1)
// keeps its digits where one token has nearly all of the probability; both
// terms of H are then sums of numbers of one sign.
//
// The best are chosen by (logit, lowest index) as one 64-bit number, so that
// they do not hang on the order in which anything arrives.
#include "logprobs.h"
#include "qk_common.h"
#include "qk_internal.h"

namespace qk {

namespace {

constexpr int kWaves = kLogpThreads / 64;
constexpr float kInf = __builtin_inff();

// Order of a logit: larger for a larger one, equal for both zeros, 1 for NaN.
__device__ __forceinline__ uint32_t key_of(float f) {
    const uint32_t b = __builtin_bit_cast(uint32_t, f + 0.0f);
    return f != f ? 1u : b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
    return k == 1u ? __builtin_nanf("") : __builtin_bit_cast(float, k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// (written out: max() of 64-bit whole numbers may go by way of floating point)
__device__ __forceinline__ uint64_t larger(uint64_t a, uint64_t b) { return a > b ? a : b; }

__device__ __forceinline__ uint64_t wave_max64(uint64_t v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint64_t u = __shfl_xor((unsigned long long)v, d);
        v = u > v ? u : v;
    }
    return v;
}
__device__ __forceinline__ float wave_fmax(float v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v = fmaxf(v, __shfl_xor(v, d));
    return v;
}
__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
    return v;
}

// What a part or a row has: its largest logit, how many are equal to it, and
// over the others the sums of exp(z) and, over all, of exp(z) z.
struct Stat {
    float m;
    double equal, s, w;
};

// Writes a row's results: a.lp, a.entropy and the best from their orders.
__device__ __forceinline__ void write_row(const LogpArgs &a, int64_t row, const Stat &t, const void *x, bool f16,
                                          const uint64_t *best, int threads) {
    const double rest = t.equal - 1.0 + t.s;   // S - 1
    const bool none = t.m == -kInf && t.s == 0.0;  // (a sum of NaN: NaN everywhere)
    const double ln = none ? 0.0 : log1p(rest);
    auto logp = [&](float v) { return none && v == v ? -kInf : (float)(((double)v - (double)t.m) * a.scale - ln); };
    if (threadIdx.x == 0 && a.entropy) a.entropy[row] = none ? 0.0f : (float)(ln - t.w / (1.0 + rest));
    for (int i = threadIdx.x; i < a.n_ids; i += threads) {
        const int id = a.ids[row * a.ld_ids + i];
        float v = __builtin_nanf("");
        if ((unsigned)id < (unsigned)a.vocab)
            v = f16 ? h2f(static_cast<const uint16_t *>(x)[row * a.ldx + id]) : static_cast<const float *>(x)[row * a.ldx + id];
        a.lp[row * a.ld_lp + i] = logp(v);
    }
    for (int i = threadIdx.x; i < a.top; i += threads) {
        const uint64_t b = best[i];
        a.best_ids[row * a.ld_best_ids + i] = (int)~(uint32_t)b;
        a.best[row * a.ld_best + i] = logp(value_of((uint32_t)(b >> 32)));
    }
}

template <int E, bool F16>
__global__ __launch_bounds__(kLogpThreads) void logp_kernel(const LogpArgs a) {
    constexpr int VEC = F16 ? 8 : 4;         // logits of a load
    __shared__ float red[4][kWaves];
    __shared__ uint64_t top_of[2][kWaves];
    __shared__ uint64_t best[kLogpMost];
    const int64_t row = blockIdx.x / (unsigned)a.parts;
    const int part = blockIdx.x - (unsigned)row * (unsigned)a.parts;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int first = part * (kLogpThreads * E);
    auto index_of = [&](int i) { return first + (i / VEC * kLogpThreads + (int)threadIdx.x) * VEC + i % VEC; };

    float x[E];
#pragma unroll
    for (int v = 0; v < E / VEC; ++v) {
        const int at = index_of(v * VEC);
        const int64_t from = row * a.ldx + at;
        if (at <= a.vocab - VEC) {
            if constexpr (F16) {
                uint32_t h[4];
                __builtin_memcpy(h, static_cast<const uint16_t *>(a.x) + from, 16);
#pragma unroll
                for (int i = 0; i < VEC; ++i) x[v * VEC + i] = h2f(h[i / 2] >> (16 * (i % 2)) & 0xFFFFu);
            } else {
                __builtin_memcpy(&x[v * VEC], static_cast<const float *>(a.x) + from, 16);
            }
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                x[v * VEC + i] = -kInf;
                if (at + i < a.vocab)
                    x[v * VEC + i] = F16 ? h2f(static_cast<const uint16_t *>(a.x)[from + i]) : static_cast<const float *>(a.x)[from + i];
            }
        }
    }

    // the largest
    float m = -kInf;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        m = fmaxf(m, x[i]);
        nan = nan || x[i] != x[i];
    }
    m = wave_fmax(m);
    if (lane == 0) red[0][wave] = m;
    const bool any_nan = __syncthreads_or(nan) != 0;
    m = red[0][0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) m = fmaxf(m, red[0][w]);

    // the sums (what lies behind the row's end counts as 0)
    float s = 0.0f, wz = 0.0f, equal = 0.0f;
    const float c = 1.4426950408889634f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const float z = (x[i] - m) * a.scale;
        const float e = __builtin_amdgcn_exp2f(z * c);
        const bool is = x[i] == m;
        equal += is && index_of(i) < a.vocab ? 1.0f : 0.0f;
        s += is ? 0.0f : e;
        wz += e > 0.0f ? e * z : 0.0f;
    }
    s = wave_sum(s);
    wz = wave_sum(wz);
    equal = wave_sum(equal);
    if (lane == 0) {
        red[1][wave] = s;
        red[2][wave] = wz;
        red[3][wave] = equal;
    }

    // the best, one after another
    if (a.top > 0) {
        auto order_of = [&](int i) {
            const int at = index_of(i);
            return at < a.vocab ? (uint64_t)key_of(x[i]) << 32 | (uint32_t)~at : 0ull;
        };
        uint64_t mine = 0;
#pragma unroll
        for (int i = 0; i < E; ++i) mine = larger(mine, order_of(i));
        for (int t = 0; t < a.top; ++t) {
            const uint64_t wm = wave_max64(mine);
            if (lane == 0) top_of[t & 1][wave] = wm;
            __syncthreads();
            uint64_t b = top_of[t & 1][0];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) b = larger(b, top_of[t & 1][w]);
            if (threadIdx.x == 0) best[t] = b;
            if (b != 0 && mine == b) {
                mine = 0;
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const uint64_t o = order_of(i);
                    if (o < b) mine = larger(mine, o);
                }
            }
        }
    }
    __syncthreads();
    Stat t{m, 0.0, 0.0, 0.0};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        t.s += (double)red[1][w];
        t.w += (double)red[2][w];
        t.equal += (double)red[3][w];
    }
    if (m == -kInf) t.s = t.w = 0.0;   // (nothing but -infinity: no sum)
    if (any_nan || m == kInf) t.s = __builtin_nan("");
    if (a.parts == 1) {
        write_row(a, row, t, a.x, F16, best, kLogpThreads);
        return;
    }
    if (threadIdx.x == 0) {
        float *out = a.stat + 4 * (int64_t)blockIdx.x;
        out[0] = t.m;
        out[1] = (float)t.equal;
        out[2] = (float)t.s;
        out[3] = (float)t.w;
    }
    if (threadIdx.x < (unsigned)a.top) a.list[(int64_t)blockIdx.x * a.top + threadIdx.x] = best[threadIdx.x];
}

// Joins the parts of a row.
constexpr int kJoinThreads = 256;
template <bool F16>
__global__ __launch_bounds__(kJoinThreads) void logp_join_kernel(const LogpArgs a) {
    constexpr int W = kJoinThreads / 64;
    __shared__ float redm[W];
    __shared__ double red[3][W];
    __shared__ uint64_t top_of[2][W];
    __shared__ uint64_t best[kLogpMost];
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const float *stat = a.stat + 4 * row * a.parts;
    float m = -kInf;
    for (int p = threadIdx.x; p < a.parts; p += kJoinThreads) m = fmaxf(m, stat[4 * p]);
    m = wave_fmax(m);
    if (lane == 0) redm[wave] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) m = fmaxf(m, redm[w]);
    Stat t{m, 0.0, 0.0, 0.0};
    for (int p = threadIdx.x; p < a.parts; p += kJoinThreads) {
        const float pm = stat[4 * p];
        const double equal = stat[4 * p + 1], s = stat[4 * p + 2], w = stat[4 * p + 3];
        if (pm == m) {
            t.equal += equal;
            t.s += s;
            t.w += w;
        } else {
            // with d = scale * (part's largest - m), exp(z) is exp(d) times the part's and z is d more
            const double d = ((double)pm - (double)m) * a.scale, f = exp(d);
            t.s += f * (equal + s);
            if (f > 0.0) t.w += f * (w + d * (equal + s));
        }
    }
    t.equal = wave_sum64(t.equal);
    t.s = wave_sum64(t.s);
    t.w = wave_sum64(t.w);
    if (lane == 0) {
        red[0][wave] = t.equal;
        red[1][wave] = t.s;
        red[2][wave] = t.w;
    }
    const uint64_t *list = a.list + row * a.parts * a.top;
    const int entries = a.parts * a.top;
    uint64_t last = ~0ull;
    for (int i = 0; i < a.top; ++i) {
        uint64_t mine = 0;
        for (int e = threadIdx.x; e < entries; e += kJoinThreads) {
            const uint64_t o = list[e];
            if (o < last) mine = larger(mine, o);
        }
        mine = wave_max64(mine);
        if (lane == 0) top_of[i & 1][wave] = mine;
        __syncthreads();
        last = top_of[i & 1][0];
#pragma unroll
        for (int w = 1; w < W; ++w) last = larger(last, top_of[i & 1][w]);
        if (threadIdx.x == 0) best[i] = last;
    }
    __syncthreads();
    t.equal = t.s = t.w = 0.0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        t.equal += red[0][w];
        t.s += red[1][w];
        t.w += red[2][w];
    }
    write_row(a, row, t, a.x, F16, best, kJoinThreads);
}

template <bool F16>
int run(const LogpArgs &a, int each, hipStream_t stream) {
    const int64_t most = max_groups(kLogpThreads) / a.parts;  // rows of one launch
    for (int64_t i = 0; i < a.n; i += most) {
        LogpArgs p = a;
        p.n = std::min(a.n - i, most);
        p.x = static_cast<const uint8_t *>(a.x) + i * a.ldx * (F16 ? 2 : 4);
        if (a.ids) p.ids = a.ids + i * a.ld_ids;
        if (a.lp) p.lp = a.lp + i * a.ld_lp;
        if (a.entropy) p.entropy = a.entropy + i;
        if (a.best) p.best = a.best + i * a.ld_best;
        if (a.best_ids) p.best_ids = a.best_ids + i * a.ld_best_ids;
        if (a.stat) p.stat = a.stat + 4 * i * a.parts;
        if (a.list) p.list = a.list + i * a.parts * a.top;
        const dim3 grid((unsigned)(p.n * a.parts)), block(kLogpThreads);
        int st = each == 8    ? launch(logp_kernel<8, F16>, grid, block, stream, p)
                 : each == 16 ? launch(logp_kernel<16, F16>, grid, block, stream, p)
                 : each == 32 ? launch(logp_kernel<32, F16>, grid, block, stream, p)
                              : launch(logp_kernel<64, F16>, grid, block, stream, p);
        if (st == QK_OK && a.parts > 1) st = launch(logp_join_kernel<F16>, dim3((unsigned)p.n), dim3(kJoinThreads), stream, p);
        if (st != QK_OK) return st;
    }
    return QK_OK;
}

}  // namespace

int launch_token_logprobs(const LogpArgs &a, bool f16, int each, hipStream_t stream) {
    return f16 ? run<true>(a, each, stream) : run<false>(a, each, stream);
}

}  // namespace qk
