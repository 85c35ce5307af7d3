// route.hip - routing of tokens to experts.
//
// One wave per token.  Lane l holds the scores of experts l*V .. l*V + V - 1
// (V = ceil(experts / 64) rounded up to a power of two), and the `used` best
// are taken one after another: each lane keeps its own best, a wave maximum
// finds the largest, the lowest lane that has it is the lowest index, and only
// that lane looks for its next best.  Values are compared as unsigned keys in
// the order of the floats, 0 for an expert that is out.
//
// The choice must not hang on the order of a sum: scores come from one
// exponential and correctly rounded divisions, and the softmax's sum is held in
// fp64 and rounded once.  Where no bias and no sum of two decides (both
// scores rise with the logit), the logits themselves are compared.
//
// Bound by the choices one after another for few tokens (1 x 128, 8 chosen: 3.1
// us, of which the launch is 1.6) and by vector instructions for many (about 700 a
// token: 4096 x 256 in 8 groups 6.9 us, 4096 x 128 4.6 us, their logits 1 us of
// traffic).  Groups that are segments of 1, 2, 4 .. lanes are scored all at
// once and ranked by counting (10.7 -> 7.0 us against a wave maximum per group).
#include <algorithm>

#include "qk_common.h"
#include "qk_internal.h"

namespace qk {

struct RouteArgs {
    const float *x, *bias;
    int32_t *ids;
    float *w;
    int64_t n, ldx, ld_ids, ldw;
    int experts, used, groups, kept, best;
    int sigmoid, renorm;
    float scale;
};

namespace {

constexpr int kRouteWaves = 4;

template <int CTRL, int ROW_MASK = 0xF>
__device__ __forceinline__ uint32_t max_dpp(uint32_t v) {
    const uint32_t u = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROW_MASK, 0xF, false);
    return u > v ? u : v;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max_dpp<0xB1>(v);
    v = max_dpp<0x4E>(v);
    v = max_dpp<0x141>(v);
    v = max_dpp<0x140>(v);
    v = max_dpp<0x142, 0xA>(v);
    v = max_dpp<0x143, 0xC>(v);
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Key of a value: larger for a larger float, equal for both zeros, 1 for NaN.
__device__ __forceinline__ uint32_t key_of(float f) {
    const uint32_t b = __builtin_bit_cast(uint32_t, f + 0.0f);
    return f != f ? 1u : b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
    return __builtin_bit_cast(float, k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// What a DPP move brings from another lane.
template <int CTRL>
__device__ __forceinline__ uint32_t from_dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}

// Key of a group's score: of its largest value, or of the sum of its two.
__device__ __forceinline__ uint32_t group_key(uint32_t k0, uint32_t k1, bool two) {
    if (!two) return k0;
    const float nan = __builtin_nanf("");
    return key_of((k0 == 1u ? nan : value_of(k0)) + (k1 == 1u ? nan : value_of(k1)));
}

template <int V>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(const RouteArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t tok = (int64_t)blockIdx.x * kRouteWaves + (threadIdx.x >> 6);
    if (tok >= a.n) return;  // (whole waves; the kernel has no barrier)
    const float *x = a.x + tok * a.ldx;
    const int e0 = lane * V;

    float p[V];       // logits, then scores
    uint32_t key[V];  // selection keys
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = e0 + i < a.experts ? x[e0 + i] : 0.0f;
    const bool by_logit = a.bias == nullptr && a.best == 1;
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = by_logit ? key_of(p[i]) : 0u;

    if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = 1.0f / (1.0f + expf(-p[i]));
    } else {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (e0 + i < a.experts) top = max(top, key_of(p[i]));
        top = wave_max(top);
        const float mx = value_of(top);
        const bool none = top <= key_of(-__builtin_inff());  // nothing above -inf (or NaN alone)
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float e = none && p[i] == p[i] ? 0.0f : expf(p[i] - mx);
            p[i] = e;
            if (e0 + i < a.experts) sum += (double)e;
        }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
        const float fs = (float)sum;
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = fs == 0.0f ? 0.0f : p[i] / fs;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (!by_logit) key[i] = key_of(a.bias != nullptr && e0 + i < a.experts ? p[i] + a.bias[e0 + i] : p[i]);
        if (e0 + i >= a.experts) key[i] = 0u;
    }

    if (a.kept < a.groups) {
        const int size = a.experts / a.groups;
        const int lanes = size / V;
        if (size % V == 0 && (lanes & (lanes - 1)) == 0) {
            // a group is a segment of 1, 2, 4 .. lanes: all groups' two largest at once
            uint32_t b0 = 0, b1 = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                b1 = max(b1, min(b0, key[i]));
                b0 = max(b0, key[i]);
            }
            auto join = [&](uint32_t o0, uint32_t o1) {
                b1 = max(max(b1, o1), min(b0, o0));
                b0 = max(b0, o0);
            };
            if (lanes > 1) join(from_dpp<0xB1>(b0), from_dpp<0xB1>(b1));
            if (lanes > 2) join(from_dpp<0x4E>(b0), from_dpp<0x4E>(b1));
            if (lanes > 4) join(from_dpp<0x141>(b0), from_dpp<0x141>(b1));
            if (lanes > 8) join(from_dpp<0x140>(b0), from_dpp<0x140>(b1));
            if (lanes > 16) join((uint32_t)__shfl_xor((int)b0, 16), (uint32_t)__shfl_xor((int)b1, 16));
            const uint32_t mine = group_key(b0, b1, a.best == 2 && size > 1);
            // its rank among the groups, of equal ones the first ahead
            const int group = lane / lanes;
            int rank = 0;
            for (int q = 0; q < a.groups; ++q) {
                const uint32_t other = (uint32_t)__builtin_amdgcn_readlane((int)mine, q * lanes);
                rank += other > mine || (other == mine && q < group) ? 1 : 0;
            }
            if (rank >= a.kept) {
#pragma unroll
                for (int i = 0; i < V; ++i) key[i] = 0u;
            }
        } else {
            uint32_t mine = 0;  // lane q: key of group q's score
            for (int q = 0; q < a.groups; ++q) {
                uint32_t b0 = 0, b1 = 0;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const uint32_t k = (unsigned)(e0 + i - q * size) < (unsigned)size ? key[i] : 0u;
                    b1 = max(b1, min(b0, k));
                    b0 = max(b0, k);
                }
                const uint32_t m0 = wave_max(b0);
                const int first = __builtin_ctzll(__ballot(b0 == m0));
                const uint32_t m1 = wave_max(lane == first ? b1 : b0);
                const uint32_t k = group_key(m0, m1, a.best == 2 && size > 1);
                if (lane == q) mine = k;
            }
            uint64_t keep = 0;
            for (int q = 0; q < a.kept; ++q) {
                const uint32_t m = wave_max(mine);
                const int first = __builtin_ctzll(__ballot(mine == m));
                keep |= 1ull << first;
                if (lane == first) mine = 0;
            }
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (e0 + i < a.experts && !(keep >> ((e0 + i) / size) & 1)) key[i] = 0u;
        }
    }

    // the best `used`, one after another; lane s keeps choice s
    int my_id = 0;
    for (int s = 0; s < a.used; ++s) {
        uint32_t b = key[0];
        int bi = 0;
#pragma unroll
        for (int i = 1; i < V; ++i)
            if (key[i] > b) {
                b = key[i];
                bi = i;
            }
        const uint32_t m = wave_max(b);
        const int first = __builtin_ctzll(__ballot(b == m));
        const int slot = __builtin_amdgcn_readlane(bi, first);
        my_id = lane == s ? first * V + slot : my_id;
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = lane == first && i == slot ? 0u : key[i];
    }
    float my_w = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float w = __shfl(p[i], my_id / V);
        my_w = my_id % V == i ? w : my_w;
    }
    if (a.renorm) {
        const float sum = wave_sum(lane < a.used ? my_w : 0.0f);
        my_w = sum == 0.0f ? 0.0f : my_w / sum;
    }
    if (lane < a.used) {
        a.ids[tok * a.ld_ids + lane] = my_id;
        a.w[tok * a.ldw + lane] = my_w * a.scale;
    }
}

}  // namespace

int launch_moe_route(const float *x, int64_t ldx, int64_t n, int64_t experts, int64_t used, bool sigmoid,
                     const float *bias, int64_t groups, int64_t kept, int64_t best, bool renorm, float scale,
                     int32_t *ids, int64_t ld_ids, float *w, int64_t ldw, hipStream_t stream) {
    const dim3 block(64 * kRouteWaves);
    constexpr int64_t most = max_groups(64 * kRouteWaves) * kRouteWaves;  // tokens
    for (int64_t tok = 0; tok < n; tok += most) {
        const int64_t part = std::min(n - tok, most);
        const RouteArgs a{x + tok * ldx, bias, ids + tok * ld_ids, w + tok * ldw, part, ldx, ld_ids, ldw,
                          (int)experts, (int)used, (int)groups, (int)kept, (int)best, sigmoid, renorm, scale};
        const dim3 grid((unsigned)((part + kRouteWaves - 1) / kRouteWaves));
        const int st = experts <= 64    ? launch(route_kernel<1>, grid, block, stream, a)
                       : experts <= 128 ? launch(route_kernel<2>, grid, block, stream, a)
                       : experts <= 256 ? launch(route_kernel<4>, grid, block, stream, a)
                       : experts <= 512 ? launch(route_kernel<8>, grid, block, stream, a)
                                        : launch(route_kernel<16>, grid, block, stream, a);
        if (st != QK_OK) return st;
    }
    return QK_OK;
}

}  // namespace qk
