// norm.hip - root-mean-square norm with the residual's addition.
//
//   s = x + residual,  y = s / sqrt(mean(s^2) + eps) * weight
//
// One read of x and residual, one write of s and y: the row stays in
// registers between the sum of squares and the scaling (rows of more than
// 16384 elements are read twice).  The sum of squares is held in fp64, which
// costs nothing beside the loads and cannot overflow, and the row's factor is
// rounded to fp32 once; where it lies outside fp32's normal range (rows of
// subnormal values without eps, rows near the largest value) the elements are
// moved by a power of two first, which leaves y's digits as they are.
//
// Bound by that traffic from about 512 rows: 2048 x 4096 fp32 to 8 bits 20.5 us
// (110 MB, 5.4 TB/s), fp16 to fp16 12.6 us (67 MB, 5.3 TB/s); below by one row's
// chain of loads, sums and stores: 1 x 4096 3.4 us, of which the launch is 1.6.
#include <algorithm>

#include "qk_common.h"
#include "qk_internal.h"

namespace qk {

struct NormArgs {
    const void *x, *r;
    const float *w;
    void *s, *y;
    int64_t ldx, ldr, lds, ldy;  // elements; QK_X8 outputs: bytes
    int64_t n;
    int k;
    double eps;
};

namespace {

typedef float f4_t __attribute__((ext_vector_type(4)));
typedef _Float16 h4_t __attribute__((ext_vector_type(4)));

// Elements c..c+3 (those below k, 0 past it).
template <typename T>
__device__ __forceinline__ f4_t load4(const T *p, int c, int k) {
    f4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c + 4 <= k) {
        T t[4];
        __builtin_memcpy(t, p + c, sizeof(t));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (float)t[i];
    } else {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (c + i < k) v[i] = (float)p[c + i];
    }
    return v;
}

// STREAM: stores past the caches.  A large call's outputs would push out what
// is still to be read (fp32 rows: 2048 x 4096 26.2 -> 22.5 us, 512 x 4096 8.8 ->
// 6.8; 256 x 4096 5.3 -> 5.0); a small call's are read by the next kernel.
template <bool STREAM, typename T>
__device__ __forceinline__ void put(T *p, const T &v) {
    if constexpr (STREAM) __builtin_nontemporal_store(v, p);
    else *p = v;
}
template <bool STREAM, typename T>
__device__ __forceinline__ void store4(T *p, int c, int k, const f4_t &v) {
    if (c + 4 <= k) {
        typedef T t4 __attribute__((ext_vector_type(4), aligned(sizeof(T))));
        t4 t;
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = (T)v[i];
        if constexpr (STREAM) __builtin_nontemporal_store(t, reinterpret_cast<t4 *>(p + c));
        else *reinterpret_cast<t4 *>(p + c) = t;
    } else {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (c + i < k) p[c + i] = (T)v[i];
    }
}

// Four elements of a 32-element block held by eight neighbouring lanes to
// 8-bit codes with the power-of-two scale that qk_mul_mat_vec_x8 takes: d =
// 2^e, e the smallest integer >= -126 with 127 * 2^e >= max|x|; d = 0 for an
// all-zero block, NaN (codes 0) for one with an infinite or NaN value.
__device__ __forceinline__ uint32_t block_codes(const f4_t &v, float &d) {
    float top = 0.0f;
    bool fine = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        top = fmaxf(top, fabsf(v[i]));
        fine = fine && fabsf(v[i]) <= 3.402823466e38f;
    }
    if (!fine) top = __builtin_inff();
    top = fmaxf(top, dpp<0xB1>(top));    // quad_perm [1,0,3,2]
    top = fmaxf(top, dpp<0x4E>(top));    // quad_perm [2,3,0,1]
    top = fmaxf(top, dpp<0x141>(top));   // row_half_mirror
    fine = top <= 3.402823466e38f;
    int ex;
    const float mant = frexpf(fine ? top : 0.0f, &ex);
    const int e = max(ex - 7 + (mant > 0.9921875f ? 1 : 0), -126);  // 127 / 128
    d = !fine ? __builtin_nanf("") : top == 0.0f ? 0.0f : ldexpf(1.0f, e);
    if (!fine) return 0;
    const float inv = ldexpf(1.0f, -e);
    // adding 1.5 * 2^23 rounds to a whole number, half to even; the low byte
    // of the sum is that number in two's complement
    uint32_t q = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        q |= (__builtin_bit_cast(uint32_t, v[i] * inv + 12582912.0f) & 0xFFu) << (8 * i);
    return q;
}

// T threads per row; R groups of four elements per thread in registers (0: no
// bound on the row, which is read twice).
template <typename XT, int YT, int T, int R, bool STREAM>
__global__ __launch_bounds__(T < 256 ? 256 : T) void rms_norm_kernel(const NormArgs a) {
    constexpr int ROWS = T < 256 ? 256 / T : 1;
    const int t = threadIdx.x % T;
    const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / T;
    if (T <= 64 && row >= a.n) return;  // (whole waves, and no barrier follows)
    const XT *x = static_cast<const XT *>(a.x) + row * a.ldx;
    const XT *r = a.r ? static_cast<const XT *>(a.r) + row * a.ldr : nullptr;
    XT *s = a.s ? static_cast<XT *>(a.s) + row * a.lds : nullptr;
    auto sum_at = [&](int c) {
        f4_t v = load4(x, c, a.k);
        if (r) {
            const f4_t u = load4(r, c, a.k);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += u[i];
        }
        return v;
    };
    double ss = 0.0;
    auto add = [&](const f4_t &v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) ss = __builtin_fma((double)v[i], (double)v[i], ss);
    };
    f4_t v[R > 0 ? R : 1];
    if constexpr (R > 0) {
#pragma unroll
        for (int i = 0; i < R; ++i) v[i] = sum_at(4 * (t + i * T));
#pragma unroll
        for (int i = 0; i < R; ++i) add(v[i]);
    } else {
        for (int64_t c = 4 * t; c < a.k; c += 4 * T) add(sum_at((int)c));
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) ss += __shfl_xor(ss, d);
    if constexpr (T > 64) {
        __shared__ double part[T / 64];
        if (t % 64 == 0) part[t / 64] = ss;
        __syncthreads();
        ss = 0.0;
#pragma unroll
        for (int i = 0; i < T / 64; ++i) ss += part[i];
    }
    const double factor = 1.0 / sqrt(ss / a.k + a.eps);
    // (selected, not branched on: the weights' loads stay ahead of this chain,
    // 1 x 4096 3.4 us; with a branch 3.6, with no such step 3.3)
    const bool above = factor > 0x1p100, below = factor < 0x1p-100;
    const float up = above ? 0x1p64f : below ? 0x1p-64f : 1.0f;
    const float f = (float)(factor * (above ? 0x1p-64 : below ? 0x1p64 : 1.0));
    auto finish = [&](int c, const f4_t &u) {
        if (c >= a.k) return;
        if (s) store4<STREAM>(s, c, a.k, u);
        f4_t y;
        f4_t w = {1.0f, 1.0f, 1.0f, 1.0f};
        if (a.w) w = load4(a.w, c, a.k);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = u[i] * up * f * w[i];
        if constexpr (YT == QK_X8) {
            // (k is a multiple of 32: eight lanes hold a block, all of it)
            uint8_t *b = static_cast<uint8_t *>(a.y) + row * a.ldy + (int64_t)(c >> 5) * 36;
            float d;
            const uint32_t q = block_codes(y, d);
            put<STREAM>(reinterpret_cast<uint32_t *>(b + 4 + (c & 31)), q);
            if ((c & 31) == 0) put<STREAM>(reinterpret_cast<float *>(b), d);
        } else if constexpr (YT == QK_F16) {
            store4<STREAM>(static_cast<_Float16 *>(a.y) + row * a.ldy, c, a.k, y);
        } else {
            store4<STREAM>(static_cast<float *>(a.y) + row * a.ldy, c, a.k, y);
        }
    };
    if constexpr (R > 0) {
#pragma unroll
        for (int i = 0; i < R; ++i) finish(4 * (t + i * T), v[i]);
    } else {
        for (int64_t c = 4 * t; c < a.k; c += 4 * T) finish((int)c, sum_at((int)c));
    }
}

template <typename XT, int YT, int T, int R, bool STREAM>
int start_parts(const NormArgs &a, hipStream_t stream) {
    constexpr int ROWS = T <= 64 ? 4 : 1, THREADS = T < 256 ? 256 : T;
    constexpr int64_t most = max_groups(THREADS) * ROWS;  // rows
    constexpr int64_t xe = sizeof(XT), ye = YT == QK_X8 ? 1 : YT == QK_F16 ? 2 : 4;
    for (int64_t row = 0; row < a.n; row += most) {
        NormArgs p = a;
        p.n = std::min(a.n - row, most);
        p.x = static_cast<const uint8_t *>(a.x) + row * a.ldx * xe;
        if (a.r) p.r = static_cast<const uint8_t *>(a.r) + row * a.ldr * xe;
        if (a.s) p.s = static_cast<uint8_t *>(a.s) + row * a.lds * xe;
        p.y = static_cast<uint8_t *>(a.y) + row * a.ldy * ye;
        const dim3 grid((unsigned)((p.n + ROWS - 1) / ROWS));
        const int st = launch(rms_norm_kernel<XT, YT, T, R, STREAM>, grid, dim3(THREADS), stream, p);
        if (st != QK_OK) return st;
    }
    return QK_OK;
}
template <typename XT, int YT, int T, int R>
int start(const NormArgs &a, hipStream_t stream) {
    if (a.n * a.k > (int64_t(1) << 20)) return start_parts<XT, YT, T, R, true>(a, stream);
    return start_parts<XT, YT, T, R, false>(a, stream);
}

template <typename XT, int YT>
int run(const NormArgs &a, hipStream_t stream) {
    const int64_t n = a.n;
    // Up to two rows per CU a row has more threads, so that the chain of one
    // thread's loads and adds is short (1 x 4096 4.5 -> 3.4 us, 256 x 4096 to
    // 8 bits 7.3 -> 5.4); beyond, fewer threads leave more rows to a CU (2048 x
    // 4096 to 8 bits 24.4 us against 26.0).
    const bool wide = n <= 2 * (int64_t)device_cus();
    if (wide && a.k <= 256) return start<XT, YT, 64, 1>(a, stream);
    if (wide && a.k <= 1024) return start<XT, YT, 256, 1>(a, stream);
    if (wide && a.k <= 4096) return start<XT, YT, 1024, 1>(a, stream);
    if (a.k <= 1024) return start<XT, YT, 64, 4>(a, stream);
    if (a.k <= 4096) return start<XT, YT, 256, 4>(a, stream);
    if (a.k <= 16384) return start<XT, YT, 1024, 4>(a, stream);
    return start<XT, YT, 1024, 0>(a, stream);
}

template <typename XT>
int by_output(int y_dtype, const NormArgs &a, hipStream_t stream) {
    switch (y_dtype) {
    case QK_F32: return run<XT, QK_F32>(a, stream);
    case QK_F16: return run<XT, QK_F16>(a, stream);
    default: return run<XT, QK_X8>(a, stream);
    }
}

}  // namespace

int launch_rms_norm(int x_dtype, const void *x, int64_t ldx, const void *residual, int64_t ldr,
                    const float *weight, double eps, int64_t n, int64_t k, void *sum, int64_t lds,
                    int y_dtype, void *y, int64_t ldy, hipStream_t stream) {
    // The least mean square of a row that is not zero is 2^-328.  A smaller eps
    // still makes a zero row zero, as which its factor has to be finite; 2^-382
    // and less are nothing to any other row.
    if (eps > 0.0) eps = std::max(eps, 0x1p-382);
    const NormArgs a{x, residual, weight, sum, y, ldx, ldr, lds, ldy, n, (int)k, eps};
    return x_dtype == QK_F16 ? by_output<_Float16>(y_dtype, a, stream) : by_output<float>(y_dtype, a, stream);
}

}  // namespace qk
