// api.hip - the C ABI: argument validation, then dispatch to the launchers.
//
// Validation happens entirely on the host before any HIP call, so every error
// path returns a status with nothing enqueued.
#include <stdint.h>
#include <stddef.h>

#include <algorithm>
#include <initializer_list>

#include "attn.h"
#include "qk.h"
#include "qk_common.h"
#include "qk_internal.h"

namespace {

constexpr int64_t kMaxDim = INT32_MAX;  // kernels index rows and columns in 32 bits

bool fmt_ok(int fmt) { return qk::block_bytes_host(fmt) != 0; }

// Half-open byte ranges [a, a+na) and [b, b+nb) intersect.
bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
    if (na == 0 || nb == 0) return false;
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x < y + nb && y < x + na;
}

// Bytes spanned by n columns of length len with stride ld (elements of size es).
size_t span_bytes(int64_t n, int64_t ld, int64_t len, size_t es) {
    if (n <= 0 || len <= 0) return 0;
    return (size_t)((n - 1) * ld + len) * es;
}

constexpr int64_t kMaxNormRow = int64_t(1) << 30;

// Strides whose products with 32-bit counts stay far below 2^63 bytes.
bool stride_ok(int64_t ld) { return ld >= 0 && ld <= (int64_t(1) << 27); }
bool ld_ok(int64_t n, int64_t ld, int64_t len) {
    return ld >= len && (n <= 1 || ld <= (int64_t(1) << 58) / (n - 1));
}

struct Range {
    const void *p;
    size_t n;
};

// `len` elements at every combination of steps i < n times stride: whether
// no two share an element (steps sorted by stride, each must clear the span
// of those below it).
struct Step {
    int64_t n, stride;
};
bool rows_disjoint(int64_t len, std::initializer_list<Step> list) {
    Step s[4];
    int count = 0;
    for (const Step &x : list)
        if (x.n > 1) s[count++] = x;
    std::sort(s, s + count, [](const Step &a, const Step &b) { return a.stride < b.stride; });
    int64_t span = len;
    for (int i = 0; i < count; ++i) {
        if (s[i].stride < span) return false;
        span += (s[i].n - 1) * s[i].stride;
    }
    return true;
}

// A cache descriptor's own fields.
int check_cache(const qk_kv_cache *cache) {
    if (cache == nullptr) return QK_ERR_INVALID_ARG;
    const qk_kv_cache &c = *cache;
    if (c.type != QK_KV_F16 && c.type != QK_KV_I8) return QK_ERR_UNSUPPORTED;
    if (c.n_pages < 1 || c.n_pages > kMaxDim || c.n_heads < 1 || c.n_heads > 65535 || c.page_size < 1 ||
        c.page_size > (1 << 20) || c.head_dim < 32 || c.head_dim > 256 || c.head_dim % 32 != 0)
        return QK_ERR_INVALID_ARG;
    const int64_t es = c.type == QK_KV_I8 ? 1 : 2;
    const int64_t strides[] = {c.page_stride, c.head_stride, c.slot_stride};
    const int64_t most = int64_t(1) << 40;
    for (int64_t s : strides)
        if (s < 0 || s > most) return QK_ERR_INVALID_ARG;
    // (the last element's place must be a number)
    const double end = (double)(c.n_pages - 1) * c.page_stride + (double)(c.n_heads - 1) * c.head_stride +
                       (double)(c.page_size - 1) * c.slot_stride;
    if (end > 9.0e15) return QK_ERR_INVALID_ARG;
    if (c.k == nullptr || c.v == nullptr) return QK_ERR_INVALID_ARG;
    if (((uintptr_t)c.k | (uintptr_t)c.v) % 16 != 0) return QK_ERR_ALIGNMENT;
    for (int64_t s : strides)
        if (s * es % 16 != 0) return QK_ERR_ALIGNMENT;
    if (c.type == QK_KV_I8) {
        if (c.k_scale == nullptr || c.v_scale == nullptr) return QK_ERR_INVALID_ARG;
        const int64_t ss[] = {c.scale_page_stride, c.scale_head_stride, c.scale_slot_stride};
        for (int64_t s : ss)
            if (s < 0 || s > most) return QK_ERR_INVALID_ARG;
        const double send = (double)(c.n_pages - 1) * c.scale_page_stride + (double)(c.n_heads - 1) * c.scale_head_stride +
                            (double)(c.page_size - 1) * c.scale_slot_stride;
        if (send > 2.0e15) return QK_ERR_INVALID_ARG;
        if (((uintptr_t)c.k_scale | (uintptr_t)c.v_scale) % 4 != 0) return QK_ERR_ALIGNMENT;
    }
    return QK_OK;
}

// The memory of a (checked) cache: keys, values, and the scales of 8 bits.
struct Ranges {
    Range r[4];
    int count;
    const Range *begin() const { return r; }
    const Range *end() const { return r + count; }
    size_t size() const { return (size_t)count; }
    const Range &operator[](size_t i) const { return r[i]; }
};
Ranges cache_ranges(const qk_kv_cache &c) {
    const size_t es = c.type == QK_KV_I8 ? 1 : 2;
    const size_t n = es * (size_t)(c.head_dim + (c.n_pages - 1) * c.page_stride + (c.n_heads - 1) * c.head_stride +
                                   (c.page_size - 1) * c.slot_stride);
    Ranges out{{{c.k, n}, {c.v, n}}, 2};
    if (c.type == QK_KV_I8) {
        const size_t s = 4 * (size_t)(1 + (c.n_pages - 1) * c.scale_page_stride + (c.n_heads - 1) * c.scale_head_stride +
                                      (c.page_size - 1) * c.scale_slot_stride);
        out.r[2] = {c.k_scale, s};
        out.r[3] = {c.v_scale, s};
        out.count = 4;
    }
    return out;
}

// The most 32-token tiles that a sequence of up to max_len tokens can have.
int64_t attn_tiles(const qk::AttnArgs &a) {
    const int64_t all = (a.max_len + qk::kAttnTile - 1) / qk::kAttnTile;
    if (a.window == 0) return all;
    return std::min<int64_t>(all, (a.sinks + qk::kAttnTile - 1) / qk::kAttnTile +
                                      (a.window + qk::kAttnTile - 1) / qk::kAttnTile + 1);
}

// Workgroups that a decode attention is split for (see attn_plan).
int64_t attn_target(const qk_kv_cache &c) { return (c.head_dim <= 128 ? 2 : 1) * (int64_t)qk::device_cus(); }

// Sizes and the split of a decode attention over the cache's length: the
// tokens of a sequence go to workgroups in chunks of `chunk_tiles` 32-token
// tiles.  The lengths are on the device, so the chunk follows from max_len:
// enough chunks to give every CU two workgroups (one where head_dim leaves room
// for one wave per SIMD), and at least one tile for each wave of a workgroup.
// Beginning and ending a chunk costs a workgroup several microseconds under
// load, so more and shorter chunks cost more than their balance gives:
// 131072 tokens of 8 x 128 in fp16 at 2 / 3 / 4 / 8 / 16 workgroups per CU 100.7 /
// 101.8 / 105 / 110 / 121 us; 64 sequences of 2048 tokens in 8 bits 57 / - / 63 / 67 /
// -, of 64..4096 tokens 75 / 74 / 74 / 73 / 74; head_dim 256, 131072 tokens of 2
// heads at 1 / 2 63 / 72.
int attn_plan(const qk_kv_cache &c, int64_t n_seqs, int64_t n_q_heads, int64_t max_len, int64_t window,
              int64_t sinks, qk::AttnArgs &a) {
    if (n_seqs < 0 || n_seqs > kMaxDim || n_q_heads < 1 || n_q_heads % c.n_heads != 0 || n_q_heads > (1 << 20) ||
        max_len < 1 || max_len > (int64_t(1) << 30) || window < 0 || sinks < 0)
        return QK_ERR_INVALID_ARG;
    a.n_seqs = (int)n_seqs;
    a.n_heads = (int)n_q_heads;
    a.n_kv = (int)c.n_heads;
    a.group = (int)(n_q_heads / c.n_heads);
    a.head_tiles = (a.group + qk::kAttnHeads - 1) / qk::kAttnHeads;
    a.n_pages = (int)c.n_pages;
    a.page_size = (int)c.page_size;
    // quotients of 30-bit numbers: with 2^s >= page_size, the product's excess
    // over t * 2^(30+s) / page_size stays below 2^(30+s) / page_size
    int s = 0;
    while ((int64_t(1) << s) < c.page_size) ++s;
    a.page_shift = 30 + s;
    a.page_magic = (uint32_t)(((uint64_t(1) << (30 + s)) + c.page_size - 1) / c.page_size);
    a.max_len = (int)max_len;
    a.window = (int)std::min<int64_t>(window, max_len);
    a.sinks = (int)std::min<int64_t>(sinks, max_len);
    if (n_seqs == 0) return QK_OK;
    const int64_t tiles = attn_tiles(a);
    const int64_t rows = n_seqs * a.n_kv * a.head_tiles;
    const int64_t target = attn_target(c);
    int64_t chunk = (tiles * rows + target - 1) / target;
    chunk = std::max<int64_t>(qk::kAttnWaves, (chunk + qk::kAttnWaves - 1) / qk::kAttnWaves * qk::kAttnWaves);
    a.chunk_tiles = (int)std::min<int64_t>(chunk, tiles);
    a.nchunks = (int)((tiles + a.chunk_tiles - 1) / a.chunk_tiles);
    if (rows * a.nchunks > kMaxDim || n_seqs * n_q_heads > kMaxDim) return QK_ERR_INVALID_ARG;
    return QK_OK;
}

size_t attn_workspace(const qk_kv_cache &c, const qk::AttnArgs &a) {
    if (a.nchunks <= 1) return 0;
    return 4 * (size_t)a.n_seqs * a.n_heads * a.nchunks * (size_t)qk::attn_part_floats((int)c.head_dim);
}

// The most that attn_workspace() asks for over calls of up to these sizes, so
// that scratch made once serves a batch that shrinks.  With r < target rows,
// chunks of at least max(kAttnWaves, tiles * r / target) tiles: a row has at
// most tiles / kAttnWaves of them rounded up, and all rows at most target + r.
// (From target rows on there is one chunk a row, and nothing to join.)
size_t attn_workspace_bound(const qk_kv_cache &c, const qk::AttnArgs &a) {
    const int64_t tiles = attn_tiles(a), row = (int64_t)a.n_kv * a.head_tiles, target = attn_target(c);
    if (tiles <= qk::kAttnWaves || row >= target) return 0;
    const int64_t seqs = std::min<int64_t>(a.n_seqs, (target - 1) / row);
    const int64_t parts = std::min(seqs * ((tiles + qk::kAttnWaves - 1) / qk::kAttnWaves), target / row + seqs);
    return 4 * (size_t)parts * a.n_heads * (size_t)qk::attn_part_floats((int)c.head_dim);
}

}  // namespace

extern "C" {

size_t qk_block_bytes(int fmt) { return (size_t)qk::block_bytes_host(fmt); }

size_t qk_row_bytes(int fmt, int64_t k) {
    if (!fmt_ok(fmt) || k < 0 || k % 32 != 0) return 0;
    return (size_t)(k / 32) * (size_t)qk::block_bytes_host(fmt);
}

const char *qk_status_string(int status) {
    switch (status) {
    case QK_OK: return "ok";
    case QK_ERR_INVALID_ARG: return "invalid argument";
    case QK_ERR_UNSUPPORTED: return "unsupported format or dtype";
    case QK_ERR_ALIGNMENT: return "misaligned pointer";
    case QK_ERR_LAUNCH: return "kernel launch failed";
    default: return "unknown status";
    }
}

int qk_version(void) { return 300; }

int qk_dequantize(int fmt, const void *w, int64_t rows, int64_t k, int out_dtype, void *out,
                  void *stream) {
    if (!fmt_ok(fmt)) return QK_ERR_UNSUPPORTED;
    if (out_dtype != QK_F32 && out_dtype != QK_F16) return QK_ERR_UNSUPPORTED;
    if (rows < 0 || k < 0 || k % 32 != 0) return QK_ERR_INVALID_ARG;
    if (rows == 0 || k == 0) return QK_OK;
    if (k > kMaxDim || rows > INT64_MAX / (k / 32)) return QK_ERR_INVALID_ARG;
    // chunks of 128 blocks are numbered in 32 bits on the device side
    if ((rows * (k / 32) + 127) / 128 > (int64_t)INT32_MAX) return QK_ERR_INVALID_ARG;
    if (w == nullptr || out == nullptr) return QK_ERR_INVALID_ARG;
    const size_t es = out_dtype == QK_F32 ? 4 : 2;
    if ((uintptr_t)w % 2 != 0 || (uintptr_t)out % es != 0) return QK_ERR_ALIGNMENT;
    const int64_t nblocks = rows * (k / 32);
    const size_t wbytes = (size_t)nblocks * qk::block_bytes_host(fmt);
    const size_t obytes = (size_t)(rows * k) * es;
    if (overlaps(w, wbytes, out, obytes)) return QK_ERR_INVALID_ARG;
    return qk::launch_dequantize(fmt, w, nblocks, out_dtype, out,
                                 static_cast<hipStream_t>(stream));
}

// Checks one GEMV problem (n already known to be 1..8); QK_OK if valid.
static int check_gemv_item(int fmt, const qk_mat_vec_item &it, int64_t n) {
    if (it.m < 0 || it.k < 0 || it.k % 32 != 0) return QK_ERR_INVALID_ARG;
    if (it.m == 0) return QK_OK;
    if (it.m > kMaxDim || it.k > kMaxDim || it.ldx < it.k || it.ldy < it.m) return QK_ERR_INVALID_ARG;
    if (it.y == nullptr || (it.k > 0 && (it.w == nullptr || it.x == nullptr))) return QK_ERR_INVALID_ARG;
    if ((uintptr_t)it.w % 2 != 0 || (uintptr_t)it.x % 4 != 0 || (uintptr_t)it.y % 4 != 0)
        return QK_ERR_ALIGNMENT;
    const size_t wbytes = (size_t)it.m * (size_t)(it.k / 32) * qk::block_bytes_host(fmt);
    const size_t xbytes = span_bytes(n, it.ldx, it.k, 4);
    const size_t ybytes = span_bytes(n, it.ldy, it.m, 4);
    if (overlaps(it.y, ybytes, it.w, wbytes) || overlaps(it.y, ybytes, it.x, xbytes))
        return QK_ERR_INVALID_ARG;
    return QK_OK;
}

int qk_mul_mat_vec(int fmt, const void *w, int64_t m, int64_t k, const float *x, int64_t n,
                   int64_t ldx, float *y, int64_t ldy, void *stream) {
    if (!fmt_ok(fmt)) return QK_ERR_UNSUPPORTED;
    if (m < 0 || k < 0 || k % 32 != 0 || n < 0 || n > 8) return QK_ERR_INVALID_ARG;
    if (m == 0 || n == 0) return QK_OK;
    const qk_mat_vec_item it{w, m, k, x, ldx, y, ldy};
    const int st = check_gemv_item(fmt, it, n);
    if (st != QK_OK) return st;
    return qk::launch_mul_mat_vec(fmt, w, m, k, x, n, ldx, y, ldy, static_cast<hipStream_t>(stream));
}

int qk_mul_mat_vec_x8(int fmt, const void *w, int64_t m, int64_t k, const float *x, int64_t n,
                      int64_t ldx, float *y, int64_t ldy, void *stream) {
    if (!fmt_ok(fmt)) return QK_ERR_UNSUPPORTED;
    if (m < 0 || k < 0 || k % 32 != 0 || n < 0 || n > 8) return QK_ERR_INVALID_ARG;
    if (m == 0 || n == 0) return QK_OK;
    const qk_mat_vec_item it{w, m, k, x, ldx, y, ldy};
    const int st = check_gemv_item(fmt, it, n);
    if (st != QK_OK) return st;
    return qk::launch_mul_mat_vec_x8(fmt, w, m, k, x, n, ldx, y, ldy, static_cast<hipStream_t>(stream));
}

int qk_mul_mat_vec_x8q(int fmt, const void *w, int64_t m, int64_t k, const void *xq, int64_t n,
                       int64_t ldx, float *y, int64_t ldy, void *stream) {
    if (!fmt_ok(fmt)) return QK_ERR_UNSUPPORTED;
    if (m < 0 || k < 0 || k % 32 != 0 || n < 0 || n > 8) return QK_ERR_INVALID_ARG;
    if (m == 0 || n == 0) return QK_OK;
    if (m > kMaxDim || k > kMaxDim) return QK_ERR_INVALID_ARG;
    const int64_t col = k / 32 * 36;
    if (n == 1) {
        ldx = col;
        ldy = m;
    }
    if (ldx < col || ldy < m) return QK_ERR_INVALID_ARG;
    if (ldx > (int64_t(1) << 58) || ldy > (int64_t(1) << 56)) return QK_ERR_INVALID_ARG;  // (spans stay below 2^62)
    if (y == nullptr || (k > 0 && (w == nullptr || xq == nullptr))) return QK_ERR_INVALID_ARG;
    if ((uintptr_t)w % 2 != 0 || (uintptr_t)xq % 4 != 0 || ldx % 4 != 0 || (uintptr_t)y % 4 != 0)
        return QK_ERR_ALIGNMENT;
    const size_t wbytes = (size_t)m * (size_t)(k / 32) * qk::block_bytes_host(fmt);
    const size_t ybytes = span_bytes(n, ldy, m, 4);
    if (overlaps(y, ybytes, w, wbytes) || overlaps(y, ybytes, xq, span_bytes(n, ldx, col, 1)))
        return QK_ERR_INVALID_ARG;
    return qk::launch_mul_mat_vec_x8q(fmt, w, m, k, xq, n, ldx, y, ldy, static_cast<hipStream_t>(stream));
}

int qk_mul_mat_vec_batched(int fmt, const qk_mat_vec_item *items, int count, int64_t n,
                           void *stream) {
    if (!fmt_ok(fmt)) return QK_ERR_UNSUPPORTED;
    if (count < 0 || count > QK_MAX_BATCH || n < 0 || n > 8) return QK_ERR_INVALID_ARG;
    if (count == 0 || n == 0) return QK_OK;
    if (items == nullptr) return QK_ERR_INVALID_ARG;
    for (int i = 0; i < count; ++i) {
        const int st = check_gemv_item(fmt, items[i], n);
        if (st != QK_OK) return st;
    }
    // no output may overlap another item's inputs or output
    for (int i = 0; i < count; ++i) {
        const qk_mat_vec_item &a = items[i];
        if (a.m == 0) continue;
        const size_t ya = span_bytes(n, a.ldy, a.m, 4);
        for (int j = 0; j < count; ++j) {
            const qk_mat_vec_item &b = items[j];
            if (j == i || b.m == 0) continue;
            const size_t wb = (size_t)b.m * (size_t)(b.k / 32) * qk::block_bytes_host(fmt);
            if (overlaps(a.y, ya, b.w, wb) || overlaps(a.y, ya, b.x, span_bytes(n, b.ldx, b.k, 4)) ||
                overlaps(a.y, ya, b.y, span_bytes(n, b.ldy, b.m, 4)))
                return QK_ERR_INVALID_ARG;
        }
    }
    return qk::launch_mul_mat_vec_batched(fmt, items, count, n, static_cast<hipStream_t>(stream));
}

// (n - 1) * ld stays below 2^58, so a sum of a few such spans (and its size
// in bytes) cannot overflow.
static bool span_fits(int64_t n, int64_t ld) {
    return n <= 1 || ld == 0 || (n - 1) <= (int64_t(1) << 58) / ld;
}

// Outputs [p, p+m) at p = i*inner_ld + o*outer_ld (i < inner_n, o < outer_n)
// are pairwise disjoint when each inner run fits inside one outer stride.
static bool nested_disjoint(int64_t m, int64_t inner_n, int64_t inner_ld, int64_t outer_n,
                            int64_t outer_ld) {
    const int64_t inner_span = inner_n > 1 ? (inner_n - 1) * inner_ld + m : m;
    return (inner_n <= 1 || inner_ld >= m) && (outer_n <= 1 || outer_ld >= inner_span);
}

int qk_mul_mat_vec_id(int fmt, const void *w, int64_t n_experts, int64_t expert_stride,
                      int64_t m, int64_t k, const int32_t *ids, int64_t ld_ids,
                      int64_t n_used, int64_t n_tokens, const float *x, int64_t x_slot,
                      int64_t x_tok, float *y, int64_t y_slot, int64_t y_tok, void *stream) {
    if (!fmt_ok(fmt)) return QK_ERR_UNSUPPORTED;
    if (m < 0 || k < 0 || k % 32 != 0 || n_used < 0 || n_tokens < 0) return QK_ERR_INVALID_ARG;
    if (m == 0 || n_used == 0 || n_tokens == 0) return QK_OK;
    if (m > kMaxDim || k > kMaxDim || n_experts < 1 || n_experts > kMaxDim ||
        n_used > kMaxDim || n_tokens > kMaxDim)
        return QK_ERR_INVALID_ARG;
    const int64_t es = n_experts > 1 ? expert_stride : 0;
    const int64_t li = n_tokens > 1 ? ld_ids : 0;
    const int64_t xs = n_used > 1 ? x_slot : 0, xt = n_tokens > 1 ? x_tok : 0;
    const int64_t ys = n_used > 1 ? y_slot : 0, yt = n_tokens > 1 ? y_tok : 0;
    if (es < 0 || li < 0 || xs < 0 || xt < 0 || ys < 0 || yt < 0) return QK_ERR_INVALID_ARG;
    if (!span_fits(n_experts, es) || !span_fits(n_tokens, li) || !span_fits(n_tokens, xt) ||
        !span_fits(n_used, xs) || !span_fits(n_tokens, yt) || !span_fits(n_used, ys))
        return QK_ERR_INVALID_ARG;
    const size_t ebytes = (size_t)m * (size_t)(k / 32) * qk::block_bytes_host(fmt);
    if (n_experts > 1 && (size_t)es < ebytes) return QK_ERR_INVALID_ARG;
    if (n_tokens > 1 && li < n_used) return QK_ERR_INVALID_ARG;
    if (n_used * n_tokens > (int64_t)INT32_MAX / ((m + 7) / 8)) return QK_ERR_INVALID_ARG;
    if (!nested_disjoint(m, n_used, ys, n_tokens, yt) && !nested_disjoint(m, n_tokens, yt, n_used, ys))
        return QK_ERR_INVALID_ARG;
    if (w == nullptr || ids == nullptr || x == nullptr || y == nullptr) return QK_ERR_INVALID_ARG;
    if ((uintptr_t)w % 2 != 0 || es % 2 != 0 || (uintptr_t)ids % 4 != 0 || (uintptr_t)x % 4 != 0 ||
        (uintptr_t)y % 4 != 0)
        return QK_ERR_ALIGNMENT;
    const size_t wbytes = (size_t)(n_experts - 1) * (size_t)es + ebytes;
    const size_t ibytes = (size_t)((n_tokens - 1) * li + n_used) * 4;
    const size_t xbytes = (size_t)((n_tokens - 1) * xt + (n_used - 1) * xs + k) * 4;
    const size_t ybytes = (size_t)((n_tokens - 1) * yt + (n_used - 1) * ys + m) * 4;
    if (overlaps(y, ybytes, w, wbytes) || overlaps(y, ybytes, ids, ibytes) ||
        overlaps(y, ybytes, x, xbytes))
        return QK_ERR_INVALID_ARG;
    return qk::launch_mul_mat_vec_id(fmt, w, n_experts, es, m, k, ids, li, n_used, n_tokens, x,
                                     xs, xt, y, ys, yt, static_cast<hipStream_t>(stream));
}

int qk_mul_mat(int fmt, const void *w, int64_t m, int64_t k, const void *x_f16, int64_t n,
               int64_t ldx, float *y, int64_t ldy, void *stream) {
    if (!fmt_ok(fmt)) return QK_ERR_UNSUPPORTED;
    if (m < 0 || k < 0 || k % 32 != 0 || n < 0) return QK_ERR_INVALID_ARG;
    if (m == 0 || n == 0) return QK_OK;
    if (m > kMaxDim || k > kMaxDim || n > kMaxDim || ldx < k || ldy < m) return QK_ERR_INVALID_ARG;
    // the tile grid is one dimension of 128 x 128 tiles
    if (((m + 127) / 128) * ((n + 127) / 128) > (int64_t)INT32_MAX) return QK_ERR_INVALID_ARG;
    if (y == nullptr || (k > 0 && (w == nullptr || x_f16 == nullptr))) return QK_ERR_INVALID_ARG;
    if ((uintptr_t)w % 2 != 0 || (uintptr_t)x_f16 % 2 != 0 || (uintptr_t)y % 4 != 0)
        return QK_ERR_ALIGNMENT;
    const size_t wbytes = (size_t)m * (size_t)(k / 32) * qk::block_bytes_host(fmt);
    const size_t xbytes = span_bytes(n, ldx, k, 2);
    const size_t ybytes = span_bytes(n, ldy, m, 4);
    if (overlaps(y, ybytes, w, wbytes) || overlaps(y, ybytes, x_f16, xbytes)) return QK_ERR_INVALID_ARG;
    return qk::launch_mul_mat(fmt, w, m, k, static_cast<const uint16_t *>(x_f16), n, ldx, y, ldy,
                              static_cast<hipStream_t>(stream));
}

int qk_rms_norm(int x_dtype, const void *x, int64_t ldx, const void *residual, int64_t ldr,
                const float *weight, double eps, int64_t n, int64_t k, void *sum, int64_t lds,
                int y_dtype, void *y, int64_t ldy, void *stream) {
    if (x_dtype != QK_F32 && x_dtype != QK_F16) return QK_ERR_UNSUPPORTED;
    if (y_dtype != QK_F32 && y_dtype != QK_F16 && y_dtype != QK_X8) return QK_ERR_UNSUPPORTED;
    const bool x8 = y_dtype == QK_X8;
    if (n < 0 || k < 1 || k > kMaxNormRow || !(eps >= 0.0) || (x8 && k % 32 != 0)) return QK_ERR_INVALID_ARG;
    if (n == 0) return QK_OK;
    if (n > kMaxDim || x == nullptr || y == nullptr) return QK_ERR_INVALID_ARG;
    const int64_t yrow = x8 ? k / 32 * 36 : k;
    if (n == 1) {
        ldx = ldr = lds = k;
        ldy = yrow;
    }
    if (!ld_ok(n, ldx, k) || !ld_ok(n, ldy, yrow) || (residual && !ld_ok(n, ldr, k)) || (sum && !ld_ok(n, lds, k)))
        return QK_ERR_INVALID_ARG;
    const size_t xe = x_dtype == QK_F32 ? 4 : 2, ye = x8 ? 1 : y_dtype == QK_F32 ? 4 : 2;
    if ((uintptr_t)x % xe != 0 || (uintptr_t)residual % xe != 0 || (uintptr_t)sum % xe != 0 ||
        (uintptr_t)weight % 4 != 0 || (uintptr_t)y % (x8 ? 4 : ye) != 0 || (x8 && ldy % 4 != 0))
        return QK_ERR_ALIGNMENT;
    const size_t xb = span_bytes(n, ldx, k, xe), yb = span_bytes(n, ldy, yrow, ye);
    const size_t rb = residual ? span_bytes(n, ldr, k, xe) : 0, sb = sum ? span_bytes(n, lds, k, xe) : 0;
    const size_t wb = weight ? (size_t)k * 4 : 0;
    if (overlaps(y, yb, x, xb) || overlaps(y, yb, residual, rb) || overlaps(y, yb, weight, wb) ||
        overlaps(y, yb, sum, sb) || overlaps(sum, sb, weight, wb))
        return QK_ERR_INVALID_ARG;
    // sum may be x or residual itself: a thread writes the elements that it read
    if (overlaps(sum, sb, x, xb) && !(sum == x && lds == ldx)) return QK_ERR_INVALID_ARG;
    if (overlaps(sum, sb, residual, rb) && !(sum == residual && lds == ldr)) return QK_ERR_INVALID_ARG;
    return qk::launch_rms_norm(x_dtype, x, ldx, residual, ldr, weight, eps, n, k, sum, lds, y_dtype, y, ldy,
                               static_cast<hipStream_t>(stream));
}

int qk_kv_store(const qk_kv_cache *cache, const float *k, int64_t k_tok, int64_t k_head,
                const float *v, int64_t v_tok, int64_t v_head, int64_t n_tokens,
                const int32_t *table, int64_t ld_table, int64_t n_seqs, int64_t max_pages,
                const int32_t *seq, const int32_t *pos, void *stream) {
    int st = check_cache(cache);
    if (st != QK_OK) return st;
    const qk_kv_cache &c = *cache;
    if (n_tokens < 0 || n_seqs < 0 || max_pages < 0) return QK_ERR_INVALID_ARG;
    if (n_tokens == 0) return QK_OK;
    if (n_tokens > kMaxDim / (2 * c.n_heads) || n_seqs > kMaxDim || max_pages > kMaxDim) return QK_ERR_INVALID_ARG;
    if (!rows_disjoint(c.head_dim, {{c.n_pages, c.page_stride}, {c.n_heads, c.head_stride}, {c.page_size, c.slot_stride}}))
        return QK_ERR_INVALID_ARG;
    if (c.type == QK_KV_I8 &&
        !rows_disjoint(1, {{c.n_pages, c.scale_page_stride}, {c.n_heads, c.scale_head_stride}, {c.page_size, c.scale_slot_stride}}))
        return QK_ERR_INVALID_ARG;
    if (k == nullptr || v == nullptr || pos == nullptr || table == nullptr) return QK_ERR_INVALID_ARG;
    if (n_seqs <= 1) ld_table = max_pages;
    if (ld_table < max_pages || !stride_ok(ld_table)) return QK_ERR_INVALID_ARG;
    if (!stride_ok(k_tok) || !stride_ok(k_head) || !stride_ok(v_tok) || !stride_ok(v_head)) return QK_ERR_INVALID_ARG;
    if (((uintptr_t)k | (uintptr_t)v | (uintptr_t)table | (uintptr_t)seq | (uintptr_t)pos) % 4 != 0) return QK_ERR_ALIGNMENT;
    const size_t kb = 4 * (size_t)(c.head_dim + (n_tokens - 1) * k_tok + (c.n_heads - 1) * k_head);
    const size_t vb = 4 * (size_t)(c.head_dim + (n_tokens - 1) * v_tok + (c.n_heads - 1) * v_head);
    const size_t tb = 4 * span_bytes(n_seqs, ld_table, max_pages, 1), ib = 4 * (size_t)n_tokens;
    for (const Range &r : cache_ranges(c)) {
        if (overlaps(r.p, r.n, k, kb) || overlaps(r.p, r.n, v, vb) || overlaps(r.p, r.n, table, tb) ||
            overlaps(r.p, r.n, pos, ib) || (seq && overlaps(r.p, r.n, seq, ib)))
            return QK_ERR_INVALID_ARG;
    }
    // Keys and values may lie between one another (pages or tokens that hold
    // both), and so may their scales: then which of the two is one more step.
    const Ranges rs = cache_ranges(c);
    for (size_t i = 0; i < rs.size(); ++i)
        for (size_t j = 0; j < i; ++j) {
            if (!overlaps(rs[i].p, rs[i].n, rs[j].p, rs[j].n)) continue;
            const uintptr_t a = (uintptr_t)rs[i].p, b = (uintptr_t)rs[j].p;
            const int64_t apart = (int64_t)(a > b ? a - b : b - a);
            const bool rows = i == 1 && j == 0, scales = i == 3 && j == 2;
            if (rows && rows_disjoint(c.head_dim, {{c.n_pages, c.page_stride}, {c.n_heads, c.head_stride},
                                                   {c.page_size, c.slot_stride}, {2, apart / (c.type == QK_KV_I8 ? 1 : 2)}}))
                continue;
            if (scales && rows_disjoint(1, {{c.n_pages, c.scale_page_stride}, {c.n_heads, c.scale_head_stride},
                                            {c.page_size, c.scale_slot_stride}, {2, apart / 4}}))
                continue;
            return QK_ERR_INVALID_ARG;
        }
    const qk::StoreArgs a{static_cast<uint8_t *>(c.k), static_cast<uint8_t *>(c.v), c.k_scale, c.v_scale, k, v,
                          table, seq, pos, c.page_stride, c.head_stride, c.slot_stride,
                          c.scale_page_stride, c.scale_head_stride, c.scale_slot_stride,
                          k_tok, k_head, v_tok, v_head, ld_table, n_tokens,
                          (int)n_seqs, (int)max_pages, (int)c.n_pages, (int)c.page_size, (int)c.n_heads, (int)c.head_dim};
    return qk::launch_kv_store(a, c.type == QK_KV_I8, static_cast<hipStream_t>(stream));
}

size_t qk_attn_decode_workspace(const qk_kv_cache *cache, int64_t n_seqs, int64_t n_q_heads,
                                int64_t max_len, int64_t window, int64_t sinks) {
    if (check_cache(cache) != QK_OK) return 0;
    qk::AttnArgs a{};
    if (attn_plan(*cache, n_seqs, n_q_heads, max_len, window, sinks, a) != QK_OK) return 0;
    return attn_workspace_bound(*cache, a);
}

int qk_attn_decode(const qk_kv_cache *cache, const float *q, int64_t q_seq, int64_t q_head,
                   int64_t n_seqs, int64_t n_q_heads, const int32_t *table, int64_t ld_table,
                   const int32_t *lens, int64_t max_len, float scale, int64_t window, int64_t sinks,
                   int y_dtype, void *y, int64_t y_seq, int64_t y_head,
                   void *workspace, size_t workspace_bytes, void *stream) {
    if (y_dtype != QK_F32 && y_dtype != QK_F16) return QK_ERR_UNSUPPORTED;
    int st = check_cache(cache);
    if (st != QK_OK) return st;
    const qk_kv_cache &c = *cache;
    qk::AttnArgs a{};
    st = attn_plan(c, n_seqs, n_q_heads, max_len, window, sinks, a);
    if (st != QK_OK) return st;
    if (n_seqs == 0) return QK_OK;
    if (q == nullptr || y == nullptr || table == nullptr || lens == nullptr) return QK_ERR_INVALID_ARG;
    const int64_t pages = (max_len + c.page_size - 1) / c.page_size;
    if (n_seqs == 1) ld_table = pages;
    if (ld_table < pages || !stride_ok(ld_table)) return QK_ERR_INVALID_ARG;
    if (!stride_ok(q_seq) || !stride_ok(q_head) || !stride_ok(y_seq) || !stride_ok(y_head)) return QK_ERR_INVALID_ARG;
    if (!rows_disjoint(c.head_dim, {{n_seqs, y_seq}, {n_q_heads, y_head}})) return QK_ERR_INVALID_ARG;
    const size_t ye = y_dtype == QK_F32 ? 4 : 2;
    if (((uintptr_t)q | (uintptr_t)table | (uintptr_t)lens) % 4 != 0 || (uintptr_t)y % ye != 0 || (uintptr_t)workspace % 16 != 0)
        return QK_ERR_ALIGNMENT;
    const size_t need = attn_workspace(c, a);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return QK_ERR_INVALID_ARG;
    const size_t qb = 4 * (size_t)(c.head_dim + (n_seqs - 1) * q_seq + (n_q_heads - 1) * q_head);
    const size_t yb = ye * (size_t)(c.head_dim + (n_seqs - 1) * y_seq + (n_q_heads - 1) * y_head);
    const Range in[] = {{q, qb}, {table, 4 * span_bytes(n_seqs, ld_table, pages, 1)}, {lens, 4 * (size_t)n_seqs}};
    if (overlaps(y, yb, workspace, need)) return QK_ERR_INVALID_ARG;
    for (const Range &r : in)
        if (overlaps(r.p, r.n, y, yb) || overlaps(r.p, r.n, workspace, need)) return QK_ERR_INVALID_ARG;
    for (const Range &r : cache_ranges(c))
        if (overlaps(r.p, r.n, y, yb) || overlaps(r.p, r.n, workspace, need)) return QK_ERR_INVALID_ARG;
    const bool i8 = c.type == QK_KV_I8;
    const int64_t es = i8 ? 1 : 2;
    a.k = static_cast<const uint8_t *>(c.k);
    a.v = static_cast<const uint8_t *>(c.v);
    a.ks = c.k_scale;
    a.vs = c.v_scale;
    a.q = q;
    a.table = table;
    a.lens = lens;
    a.y = y;
    a.part = static_cast<float *>(workspace);
    a.page_stride = c.page_stride * es;
    a.head_stride = c.head_stride * es;
    a.slot_stride = c.slot_stride * es;
    a.sc_page = c.scale_page_stride;
    a.sc_head = c.scale_head_stride;
    a.sc_slot = c.scale_slot_stride;
    a.q_seq = q_seq;
    a.q_head = q_head;
    a.y_seq = y_seq;
    a.y_head = y_head;
    a.ld_table = ld_table;
    a.qscale = (float)((double)scale * 1.4426950408889634);
    a.out_f16 = y_dtype == QK_F16;
    // sub-tiles of 16 tokens in one page, their rows within 32-bit offsets
    const bool tiled = c.page_size % 16 == 0 && a.slot_stride < (int64_t(1) << 26) && (!i8 || c.scale_slot_stride == 1);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return i8 ? qk::attn_decode_run<true>(a, (int)c.head_dim, tiled, s)
              : qk::attn_decode_run<false>(a, (int)c.head_dim, tiled, s);
}

int qk_moe_route(const float *logits, int64_t ldx, int64_t n_tokens, int64_t n_experts, int64_t n_used,
                 int score, const float *bias, int64_t n_groups, int64_t topk_groups, int64_t group_top,
                 int renorm, float scale, int32_t *ids, int64_t ld_ids, float *weights, int64_t ldw, void *stream) {
    if (score != QK_SOFTMAX && score != QK_SIGMOID) return QK_ERR_UNSUPPORTED;
    if (n_tokens < 0 || n_experts < 1 || n_experts > 1024 || n_groups < 1 || n_groups > 64 ||
        n_experts % n_groups != 0 || topk_groups < 1 || topk_groups > n_groups || group_top < 1 || group_top > 2 ||
        n_used < 1 || n_used > 64 || n_used > topk_groups * (n_experts / n_groups))
        return QK_ERR_INVALID_ARG;
    if (n_tokens == 0) return QK_OK;
    if (n_tokens > kMaxDim || logits == nullptr || ids == nullptr || weights == nullptr) return QK_ERR_INVALID_ARG;
    if (n_tokens == 1) {
        ldx = n_experts;
        ld_ids = ldw = n_used;
    }
    if (!ld_ok(n_tokens, ldx, n_experts) || !ld_ok(n_tokens, ld_ids, n_used) || !ld_ok(n_tokens, ldw, n_used))
        return QK_ERR_INVALID_ARG;
    if (((uintptr_t)logits | (uintptr_t)bias | (uintptr_t)ids | (uintptr_t)weights) % 4 != 0) return QK_ERR_ALIGNMENT;
    const size_t xb = span_bytes(n_tokens, ldx, n_experts, 4), bb = bias ? (size_t)n_experts * 4 : 0;
    const size_t ib = span_bytes(n_tokens, ld_ids, n_used, 4), wb = span_bytes(n_tokens, ldw, n_used, 4);
    if (overlaps(ids, ib, logits, xb) || overlaps(weights, wb, logits, xb) || overlaps(ids, ib, bias, bb) ||
        overlaps(weights, wb, bias, bb) || overlaps(ids, ib, weights, wb))
        return QK_ERR_INVALID_ARG;
    return qk::launch_moe_route(logits, ldx, n_tokens, n_experts, n_used, score == QK_SIGMOID, bias, n_groups,
                                topk_groups, group_top, renorm != 0, scale, ids, ld_ids, weights, ldw,
                                static_cast<hipStream_t>(stream));
}

}  // extern "C"
