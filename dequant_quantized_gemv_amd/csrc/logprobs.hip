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
//
// Many rows are bound by reading the logits once: 2048 of 32000 in fp32 51 us without
// the best (262 MB, 5.1 TB/s), 54 with 5 of them, 66 with 64.  In fp16 44, which is
// half the bytes and the same instructions: 22 a logit with everything, 22 million of
// the waves', which are 36 us of four cycles each on 1024 SIMDs (two workgroups of
// 1024 lanes share a CU, so one's loads meet the other's sums).  A row of more than 32768
// logits takes a second launch (512 x 131072 in fp32 with 5 best 59 us, 4.6 TB/s; 64 x 131072
// with 20 best 20).  A single row is a chain of latencies: load, two exchanges between
// waves, candidates, 10 us.
#include <type_traits>

#include "logprobs.h"
#include "qk_common.h"
#include "qk_internal.h"

namespace qk {

namespace {

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

// Largest of a wave's numbers, to all of its lanes.
template <int CTRL, int ROW_MASK = 0xF>
__device__ __forceinline__ uint32_t max_dpp(uint32_t v) {
    const uint32_t u = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROW_MASK, 0xF, false);
    return u > v ? u : v;
}
__device__ __forceinline__ uint32_t wave_max32(uint32_t v) {
    v = max_dpp<0xB1>(v);
    v = max_dpp<0x4E>(v);
    v = max_dpp<0x141>(v);
    v = max_dpp<0x140>(v);
    v = max_dpp<0x142, 0xA>(v);
    v = max_dpp<0x143, 0xC>(v);
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
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

// The i-th token asked for (-1 behind the last) and its logit.
__device__ __forceinline__ int asked_id(const LogpArgs &a, int64_t row, int i) {
    return i < a.n_ids ? a.ids[row * a.ld_ids + i] : -1;
}
__device__ __forceinline__ float asked_logit(const LogpArgs &a, int64_t row, bool f16, int id) {
    if ((unsigned)id >= (unsigned)a.vocab) return __builtin_nanf("");
    return f16 ? h2f(static_cast<const uint16_t *>(a.x)[row * a.ldx + id]) : static_cast<const float *>(a.x)[row * a.ldx + id];
}

// Writes a row's results: a.lp, a.entropy and the best from their orders.
__device__ __forceinline__ void write_row(const LogpArgs &a, int64_t row, const Stat &t, float asked, bool f16,
                                          const uint64_t *best, int threads) {
    const double rest = t.equal - 1.0 + t.s;   // S - 1
    const bool none = t.m == -kInf && t.s == 0.0;  // (a sum of NaN: NaN everywhere)
    const double ln = none ? 0.0 : log1p(rest);
    auto logp = [&](float v) { return none && v == v ? -kInf : (float)(((double)v - (double)t.m) * a.scale - ln); };
    if (threadIdx.x == 0 && a.entropy) a.entropy[row] = none ? 0.0f : (float)(ln - t.w / (1.0 + rest));
    for (int i = threadIdx.x; i < a.n_ids; i += threads) {
        a.lp[row * a.ld_lp + i] = logp(asked);
        asked = asked_logit(a, row, f16, asked_id(a, row, i + threads));
    }
    for (int i = threadIdx.x; i < a.top; i += threads) {
        const uint64_t b = best[i];
        a.best_ids[row * a.ld_best_ids + i] = (int)~(uint32_t)b;
        a.best[row * a.ld_best + i] = logp(value_of((uint32_t)(b >> 32)));
    }
}

// The best of a list in LDS by counting: an entry has as many ahead of it as
// are larger.  Sixteen lanes count for one entry.
template <int CTRL>
__device__ __forceinline__ int add_dpp(int v) { return v + __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, false); }
__device__ __forceinline__ void rank_list(const uint64_t *list, int n, int top, uint64_t *best, int threads) {
    for (int i = threadIdx.x >> 4; i < n; i += threads >> 4) {
        const uint64_t mine = list[i];
        int rank = 0;
        for (int k = threadIdx.x & 15; k < n; k += 16) rank += list[k] > mine ? 1 : 0;
        rank = add_dpp<0x140>(add_dpp<0x141>(add_dpp<0x4E>(add_dpp<0xB1>(rank))));
        if ((threadIdx.x & 15) == 0 && rank < top) best[rank] = mine;
    }
}

template <int T, int E, bool F16>
__global__ __launch_bounds__(T, 8) void logp_kernel(const LogpArgs a) {
    constexpr int VEC = F16 ? 8 : 4;         // logits of a load
    constexpr int STEP = T * VEC;            // of the workgroup's
    constexpr int kWaves = T / 64;
    __shared__ float red[2][kWaves];
    __shared__ uint32_t tops[kWaves], lows[kWaves], found, equals;
    __shared__ uint64_t top_of[2][kWaves];
    __shared__ uint64_t best[kLogpTop], list[kLogpList];
    const int64_t row = blockIdx.x / (unsigned)a.parts;
    const int part = blockIdx.x - (unsigned)row * (unsigned)a.parts;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int first = part * (T * E);
    typedef std::conditional_t<F16, uint16_t, float> logit_t;
    const logit_t *from = static_cast<const logit_t *>(a.x) + row * a.ldx + first;
    const int length = a.vocab - first;
    // Vector v of a thread: a step that the part does not fill is read from no
    // further than the row's last vector (which may begin in the part before),
    // what that repeats counting as -infinity.
    auto vector_at = [&](int v) {
        const int at = v * STEP + (int)threadIdx.x * VEC;
        return a.vocab >= VEC ? min(at, length - VEC) : at;
    };
    auto index_of = [&](int i) { return vector_at(i / VEC) + i % VEC; };

    // what is asked for is read ahead: the id before the row, its logit with it
    const int id = a.parts == 1 ? asked_id(a, row, threadIdx.x) : -1;
    float x[E];
    if (a.vocab >= VEC) {
        // (all loads in one block: none waits for another)
        uint32_t h[F16 ? E / 2 : 1];
#pragma unroll
        for (int v = 0; v < E / VEC; ++v) {
            if constexpr (F16) __builtin_memcpy(&h[v * VEC / 2], from + vector_at(v), 16);
            else __builtin_memcpy(&x[v * VEC], from + vector_at(v), 16);
        }
        if constexpr (F16) {
#pragma unroll
            for (int i = 0; i < E; ++i) x[i] = h2f(h[i / 2] >> (16 * (i % 2)) & 0xFFFFu);
        }
        if (length < T * E) {
#pragma unroll
            for (int v = 0; v < E / VEC; ++v) {
                const int twice = v * STEP + (int)threadIdx.x * VEC - vector_at(v);   // read before
#pragma unroll
                for (int i = 0; i < VEC; ++i) x[v * VEC + i] = i >= twice ? x[v * VEC + i] : -kInf;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = -kInf;
        if (threadIdx.x == 0) {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (i < length) x[i] = F16 ? h2f((uint16_t)from[i]) : (float)from[i];
        }
    }
    const float asked = asked_logit(a, row, F16, id);
    if (threadIdx.x == 0) found = equals = 0;

    // The largest; and a value that at least `top` of the part are not below, from
    // the r largest of each wave's lanes' largest, r a wave's share of `top`: the
    // `top`-th of all waves' largest where r is 1, else the least of the waves' r-th
    // (which leaves more candidates, but ranking r > 1 of each wave costs more:
    // 2048 rows of 32000 with 5 / 20 / 64 best 56 / 64 / 85 us ranked, 62 / 64 / 68 by the least).
    float m = x[0];
#pragma unroll
    for (int i = 1; i < E; ++i) m = __builtin_elementwise_maximum(m, x[i]);   // (NaN beside a NaN)
    const bool nan = m != m;
    uint32_t mine = key_of(m);
    const uint32_t mine_most = wave_max32(mine);
    uint32_t low = mine_most;
    for (int k = kWaves; k < a.top; k += kWaves) {
        if (lane == __builtin_ctzll(__ballot(mine == low))) mine = 0;
        low = wave_max32(mine);
    }
    if (lane == 0) {
        tops[wave] = mine_most;
        lows[wave] = low;
    }
    const bool any_nan = __syncthreads_or(nan) != 0;
    const uint32_t v = tops[lane % kWaves];
    const uint32_t most = wave_max32(v);
    if (a.top <= kWaves) {
        int rank = 0;
#pragma unroll
        for (int k = 0; k < kWaves; ++k) {
            const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)v, k);
            rank += o > v || (o == v && k < lane) ? 1 : 0;
        }
        low = (uint32_t)__builtin_amdgcn_readlane((int)v, __builtin_ctzll(__ballot(rank == max(a.top, 1) - 1)));
    } else {
        low = ~wave_max32(~lows[lane % kWaves]);
    }
    m = value_of(most);

    // The sums, in log2, of which nothing below 2^-300 counts (what is masked or
    // behind the row's end is infinitely low).
    float s = 0.0f, wz = 0.0f;
    int equal = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const float z = fmaxf((x[i] - m) * a.scale2, -300.0f);
        const float e = __builtin_amdgcn_exp2f(z);
        const bool is = x[i] == m;
        equal += is ? 1 : 0;
        s += is ? 0.0f : e;
        wz = __builtin_fmaf(e, z, wz);
    }
    s = wave_sum(s);
    wz = wave_sum(wz);
    if (equal > 0) atomicAdd(&equals, (uint32_t)equal);
    if (lane == 0) {
        red[0][wave] = s;
        red[1][wave] = wz;
    }
    if (a.top > 0) {
        auto order_of = [&](float v, int at) { return (uint64_t)key_of(v) << 32 | (uint32_t)~(first + at); };
        // those not below are few, whatever the order in which they are found
        const bool few = !any_nan && low > key_of(-kInf);
        if (few && mine_most >= low) {
            const float least = value_of(low);
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (x[i] >= least) {
                    const uint32_t n = atomicAdd(&found, 1u);
                    if (n < kLogpList) list[n] = order_of(x[i], index_of(i));
                }
        }
        __syncthreads();
        const uint32_t n = found;
        if (few && n <= kLogpList) {
            rank_list(list, (int)n, a.top, best, T);
        } else {
            // many equal ones, few logits at all, or NaN: one after another, read again
            const int end = min(length, T * E);
            auto next = [&](uint64_t below) {
                uint64_t mine = 0;
#pragma unroll 1
                for (int at = threadIdx.x; at < end; at += T) {
                    const uint64_t o = order_of(F16 ? h2f((uint16_t)from[at]) : (float)from[at], at);
                    if (o < below) mine = larger(mine, o);
                }
                return mine;
            };
            uint64_t mine = next(~0ull);
#pragma unroll 1
            for (int t = 0; t < a.top; ++t) {
                const uint64_t wm = wave_max64(mine);
                if (lane == 0) top_of[t & 1][wave] = wm;
                __syncthreads();
                uint64_t b = top_of[t & 1][0];
                for (int w = 1; w < kWaves; ++w) b = larger(b, top_of[t & 1][w]);
                if (threadIdx.x == 0) best[t] = b;
                if (b != 0 && mine == b) mine = next(b);
            }
        }
    }
    __syncthreads();
    // (waves without a result to write are done: the logarithm in fp64 costs more than the sums)
    if ((int)(threadIdx.x & ~63u) >= max(1, max(a.parts == 1 ? a.n_ids : 0, a.top))) return;
    Stat t{m, (double)equals, 0.0, 0.0};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        t.s += (double)red[0][w];
        t.w += (double)red[1][w];
    }
    t.w *= 0.6931471805599453;
    if (m == -kInf) t.s = t.w = 0.0;   // (nothing but -infinity: no sum)
    if (any_nan || m == kInf) t.s = __builtin_nan("");
    if (a.parts == 1) {
        write_row(a, row, t, asked, F16, best, T);
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
constexpr int kJoinThreads = 512;
template <bool F16>
__global__ __launch_bounds__(kJoinThreads) void logp_join_kernel(const LogpArgs a) {
    constexpr int W = kJoinThreads / 64;
    __shared__ float redm[W];
    __shared__ double red[3][W];
    __shared__ uint64_t top_of[2][W];
    __shared__ uint64_t best[kLogpTop], list[kLogpList];
    __shared__ uint32_t found;
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const float asked = asked_logit(a, row, F16, asked_id(a, row, threadIdx.x));
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
    // No fewer than `top` are not below the largest of the parts' last ones, nor
    // below the least of the parts' r-th, r a part's share of `top`.
    if (a.top > 0) {
        const uint64_t *all = a.list + row * a.parts * a.top;
        const int entries = a.parts * a.top;
        const int share = (a.top + a.parts - 1) / a.parts - 1;
        uint64_t low = 0, not_least = 0;
        for (int p = threadIdx.x; p < a.parts; p += kJoinThreads) {
            low = larger(low, all[p * a.top + a.top - 1]);
            not_least = larger(not_least, ~all[p * a.top + share]);
        }
        low = wave_max64(low);
        not_least = wave_max64(not_least);
        if (lane == 0) {
            top_of[0][wave] = low;
            top_of[1][wave] = not_least;
        }
        if (threadIdx.x == 0) found = 0;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w) {
            low = larger(low, top_of[0][w]);
            not_least = larger(not_least, top_of[1][w]);
        }
        low = larger(low, ~not_least);
        for (int e = threadIdx.x; e < entries; e += kJoinThreads) {
            const uint64_t o = all[e];
            if (o >= low && o != 0) {
                const uint32_t at = atomicAdd(&found, 1u);
                if (at < kLogpList) list[at] = o;
            }
        }
        __syncthreads();
        const uint32_t n = found;
        if (n <= kLogpList) {
            rank_list(list, (int)n, a.top, best, kJoinThreads);
        } else {
            uint64_t last = ~0ull;
#pragma unroll 1
            for (int i = 0; i < a.top; ++i) {
                uint64_t mine = 0;
                for (int e = threadIdx.x; e < entries; e += kJoinThreads) {
                    const uint64_t o = all[e];
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
        }
    }
    __syncthreads();
    if ((int)(threadIdx.x & ~63u) >= max(1, max(a.n_ids, a.top))) return;
    t.equal = t.s = t.w = 0.0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        t.equal += red[0][w];
        t.s += red[1][w];
        t.w += red[2][w];
    }
    write_row(a, row, t, asked, F16, best, kJoinThreads);
}

template <bool F16>
int run(const LogpArgs &a, const LogpSplit &split, hipStream_t stream) {
    const int64_t most = max_groups(split.threads) / a.parts;  // rows of one launch
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
        const dim3 grid((unsigned)(p.n * a.parts)), block(split.threads);
        int st = split.threads == 64    ? launch(logp_kernel<64, 32, F16>, grid, block, stream, p)
                 : split.threads == 256 ? launch(logp_kernel<256, 32, F16>, grid, block, stream, p)
                 : split.each == 8      ? launch(logp_kernel<1024, 8, F16>, grid, block, stream, p)
                 : split.each == 16     ? launch(logp_kernel<1024, 16, F16>, grid, block, stream, p)
                                        : launch(logp_kernel<1024, 32, F16>, grid, block, stream, p);
        if (st == QK_OK && a.parts > 1) st = launch(logp_join_kernel<F16>, dim3((unsigned)p.n), dim3(kJoinThreads), stream, p);
        if (st != QK_OK) return st;
    }
    return QK_OK;
}

}  // namespace

int launch_token_logprobs(const LogpArgs &a, bool f16, const LogpSplit &split, hipStream_t stream) {
    return f16 ? run<true>(a, split, stream) : run<false>(a, split, stream);
}

}  // namespace qk
