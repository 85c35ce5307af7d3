// kv_pages.hip - whole pages of a cache: copying them, and the page tables of
// sequences that fork, grow, are dropped or packed together.
//
// A table is all the state there is.  A page is held by the rows whose tokens
// lie in it and free where none does; both calls that change tables work that
// out anew from the rows, as one bit per page (a second bit: held twice), so
// there are no counts that a lost call could leave wrong.  Which free page a
// request takes follows from ranks (prefix sums over the bits in the order of
// pages, and over the requests in the order of rows), never from the order in
// which atomics arrive.
#include <algorithm>

#include "kv_pages.h"
#include "qk_common.h"
#include "qk_internal.h"

namespace qk {

namespace {

typedef uint32_t u4_t __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// copy
// ---------------------------------------------------------------------------

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;    // pieces of a thread

// Bytes of a piece: 16 where a plane's runs begin and end at multiples of 16.
__host__ __device__ inline int piece_of(const CopyPlane &p) {
    const uint64_t all = (uint64_t)(uintptr_t)p.base | (uint64_t)p.page_stride | (uint64_t)p.outer_stride |
                         (uint64_t)p.inner_stride | (uint64_t)p.bytes | p.run;
    return all % 16 == 0 ? 16 : 4;
}
__host__ __device__ inline int64_t copy_chunks(const CopyPlane &p) {
    const int64_t chunk = (int64_t)piece_of(p) * kCopyThreads * kCopyUnroll;
    return (p.bytes + chunk - 1) / chunk;
}

// A workgroup copies one chunk of one plane of one page.
__device__ __forceinline__ int64_t run_offset(const CopyPlane &p, int64_t at) {
    if (p.run == 0) return at;
    if (p.bytes <= INT32_MAX) {
        const uint32_t r = (uint32_t)at / p.run, o = r / p.inner;
        return (int64_t)o * p.outer_stride + (int64_t)(r - o * p.inner) * p.inner_stride + (uint32_t)at - r * p.run;
    }
    const int64_t r = at / p.run, o = r / p.inner;
    return o * p.outer_stride + (r - o * p.inner) * p.inner_stride + at - r * p.run;
}

template <typename PIECE>
__device__ __forceinline__ void copy_chunk(const CopyPlane &p, int from, int to, int64_t chunk) {
    PIECE x[kCopyUnroll];
    int64_t off[kCopyUnroll];
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u) {
        const int64_t at = ((chunk * kCopyUnroll + u) * kCopyThreads + threadIdx.x) * (int64_t)sizeof(PIECE);
        off[u] = at < p.bytes ? run_offset(p, at) : -1;
        if (off[u] >= 0) x[u] = *reinterpret_cast<const PIECE *>(p.base + from * p.page_stride + off[u]);
    }
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u)
        if (off[u] >= 0) *reinterpret_cast<PIECE *>(p.base + to * p.page_stride + off[u]) = x[u];
}

__global__ __launch_bounds__(kCopyThreads) void kv_copy_kernel(const CopyArgs a, const int chunks) {
    const int64_t pair = blockIdx.x / (unsigned)chunks;
    int64_t c = blockIdx.x - pair * chunks;
    const int from = a.src[pair], to = a.dst[pair];
    if ((unsigned)from >= (unsigned)a.n_pages || (unsigned)to >= (unsigned)a.n_pages || from == to) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i >= a.planes) return;
        const CopyPlane &p = a.plane[i];
        const int64_t n = copy_chunks(p);
        if (c < n) {
            if (piece_of(p) == 16) copy_chunk<u4_t>(p, from, to, c);
            else copy_chunk<uint32_t>(p, from, to, c);
            return;
        }
        c -= n;
    }
}

// ---------------------------------------------------------------------------
// tables
// ---------------------------------------------------------------------------

constexpr int kPlanThreads = 1024;

// Exclusive prefix sum over the workgroup's threads; `total` to all of them.
__device__ __forceinline__ int block_scan(int v, int &total, int (&sums)[kPlanThreads / 64]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int x = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int y = __shfl_up(x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();  // (the last call's sums are read)
    if (lane == 63) sums[wave] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 64; ++w) {
        before += w < wave ? sums[w] : 0;
        all += sums[w];
    }
    total = all;
    return before + x - v;
}

__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; }

// Tokens of a row with a place for `room`.
__device__ __forceinline__ int tokens_of(int n, int64_t room) { return n < 0 ? 0 : n > room ? (int)room : n; }
__device__ __forceinline__ int pages_of(int tokens, int page_size) {
    return (int)(((int64_t)tokens + page_size - 1) / page_size);
}

struct Row {
    int parent;        // row of the old table, or one outside it
    int had, has;      // tokens in the old row; tokens that the new one has room for
    int kept, want;    // pages taken over; pages of the new row
};

__device__ __forceinline__ Row fork_row(const ForkArgs &a, int i) {
    Row r;
    r.parent = a.parent ? a.parent[i] : i;
    const bool is = (unsigned)r.parent < (unsigned)a.n_rows;
    const int64_t room_in = (int64_t)a.in_pages * a.page_size, room = (int64_t)a.out_pages * a.page_size;
    r.had = is ? tokens_of(a.lens[r.parent], room_in) : 0;
    r.has = tokens_of(a.new_lens[i], room);
    r.kept = pages_of(min(r.had, r.has), a.page_size);
    r.want = pages_of(r.has, a.page_size);
    return r;
}

__device__ __forceinline__ int compact_kept(const CompactArgs &a, int i) {
    return pages_of(tokens_of(a.lens[i], (int64_t)a.max_pages * a.page_size), a.page_size);
}

__global__ __launch_bounds__(256) void clear_kernel(uint32_t *p, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0;
}

__global__ __launch_bounds__(256) void fork_mark_kernel(const ForkArgs a) {
    uint32_t *held = a.ws, *twice = held + page_words(a.n_pages);
    for (int i = blockIdx.x; i < a.n_new; i += gridDim.x) {
        const Row r = fork_row(a, i);
        const int32_t *row = a.table + r.parent * a.ld_table;  // (read only where kept > 0: a row that is there)
        for (int j = threadIdx.x; j < r.kept; j += 256) {
            const int p = row[j];
            if ((unsigned)p >= (unsigned)a.n_pages) continue;
            const uint32_t bit = 1u << (p & 31);
            if (atomicOr(&held[p >> 5], bit) & bit) atomicOr(&twice[p >> 5], bit);
        }
    }
}

// The requests before each row, then the free pages in ascending order, as
// many as are asked for.
__global__ __launch_bounds__(kPlanThreads) void fork_plan_kernel(const ForkArgs a) {
    __shared__ int sums[kPlanThreads / 64];
    const int words = (int)page_words(a.n_pages);
    const uint32_t *held = a.ws, *twice = held + words;
    int *list = reinterpret_cast<int *>(a.ws + 2 * words), *first = list + a.n_pages;
    int asked = 0;
    for (int i0 = 0; i0 < a.n_new; i0 += kPlanThreads) {
        const int i = i0 + threadIdx.x;
        int need = 0;
        if (i < a.n_new) {
            const Row r = fork_row(a, i);
            need = r.want - min(r.kept, r.want);
            if (r.has > r.had && r.had % a.page_size != 0) {
                const int p = a.table[r.parent * a.ld_table + r.had / a.page_size];
                if ((unsigned)p < (unsigned)a.n_pages) need += twice[p >> 5] >> (p & 31) & 1;
            }
        }
        int total;
        const int before = block_scan(need, total, sums);
        if (i < a.n_new) first[i] = asked + before;
        asked += total;
    }
    int found = 0;
    for (int w0 = 0; w0 < words && found < asked; w0 += kPlanThreads) {
        const int w = w0 + threadIdx.x;
        uint32_t free = w < words ? ~held[w] & low_bits(min(32, a.n_pages - 32 * w)) : 0u;
        int total;
        int rank = found + block_scan(__popc(free), total, sums);
        for (; free != 0 && rank < asked; ++rank) {
            list[rank] = 32 * w + __builtin_ctz(free);
            free &= free - 1;
        }
        found += total;
    }
    if (threadIdx.x == 0) {
        first[a.n_new] = asked;
        first[a.n_new + 1] = found;
        *a.missing = max(0, asked - found);
    }
}

__global__ __launch_bounds__(256) void fork_write_kernel(const ForkArgs a) {
    const int *list = reinterpret_cast<const int *>(a.ws + 2 * page_words(a.n_pages)), *first = list + a.n_pages;
    const int found = first[a.n_new + 1];
    for (int i = blockIdx.x; i < a.n_new; i += gridDim.x) {
        const Row r = fork_row(a, i);
        const int rank = first[i];
        // (a copied page is the one request that does not extend the row)
        const int copied = first[i + 1] - rank > r.want - min(r.kept, r.want) ? r.had / a.page_size : -1;
        const int32_t *row = a.table + r.parent * a.ld_table;
        for (int j = threadIdx.x; j < a.out_pages; j += 256) {
            int p = -1;
            if (j < r.kept) p = row[j];
            const int request = j == copied ? rank : j >= r.kept && j < r.want ? rank + (copied >= 0) + j - r.kept : -1;
            if (request >= 0) {
                const int got = request < found ? list[request] : -1;
                if (j == copied) {
                    a.src[i] = got >= 0 ? p : -1;
                    a.dst[i] = got;
                }
                p = got;
            }
            a.out[i * a.ld_out + j] = p;
        }
        if (copied < 0 && threadIdx.x == 0) a.src[i] = a.dst[i] = -1;
    }
}

__global__ __launch_bounds__(256) void compact_mark_kernel(const CompactArgs a) {
    for (int i = blockIdx.x; i < a.n_rows; i += gridDim.x) {
        const int kept = compact_kept(a, i);
        for (int j = threadIdx.x; j < kept; j += 256) {
            const int p = a.table[i * a.ld_table + j];
            if ((unsigned)p < (unsigned)a.n_pages) atomicOr(&a.ws[p >> 5], 1u << (p & 31));
        }
    }
}

// Live pages below page p.
__device__ __forceinline__ int live_below(const uint32_t *held, const int *before, int p) {
    return before[p >> 5] + __popc(held[p >> 5] & low_bits(p & 31));
}

// The live pages before each word, then which pages move where: the m-th live
// page from n on (n = the number of live pages) to the m-th free one below n.
__global__ __launch_bounds__(kPlanThreads) void compact_plan_kernel(const CompactArgs a) {
    __shared__ int sums[kPlanThreads / 64];
    const int words = (int)page_words(a.n_pages);
    const uint32_t *held = a.ws;
    int *before = reinterpret_cast<int *>(a.ws + words);
    int n = 0;
    for (int w0 = 0; w0 < words; w0 += kPlanThreads) {
        const int w = w0 + threadIdx.x;
        int total;
        const int b = block_scan(w < words ? __popc(held[w]) : 0, total, sums);
        if (w < words) before[w] = n + b;
        n += total;
    }
    __syncthreads();
    const int stay = n < a.n_pages ? live_below(held, before, n) : n;
    for (int w = threadIdx.x; w < words; w += kPlanThreads) {
        const uint32_t mask = low_bits(min(32, a.n_pages - 32 * w));
        const uint32_t below = 32 * w >= n ? 0u : low_bits(n - 32 * w);   // pages below n
        uint32_t moved = held[w] & ~below;
        for (int m = max(before[w] - stay, 0); moved != 0; ++m, moved &= moved - 1) a.src[m] = 32 * w + __builtin_ctz(moved);
        uint32_t hole = ~held[w] & below & mask;
        for (int m = 32 * w - before[w]; hole != 0; ++m, hole &= hole - 1) a.dst[m] = 32 * w + __builtin_ctz(hole);
    }
    for (int m = n - stay + threadIdx.x; m < a.n_pages / 2; m += kPlanThreads) a.src[m] = a.dst[m] = -1;
    if (threadIdx.x == 0) {
        *a.live = n;
        before[words] = n;
        before[words + 1] = stay;
    }
}

__global__ __launch_bounds__(256) void compact_write_kernel(const CompactArgs a) {
    const int words = (int)page_words(a.n_pages);
    const int *before = reinterpret_cast<const int *>(a.ws + words);
    const int n = before[words], stay = before[words + 1];
    for (int i = blockIdx.x; i < a.n_rows; i += gridDim.x) {
        const int kept = compact_kept(a, i);
        for (int j = threadIdx.x; j < a.max_pages; j += 256) {
            int p = -1;
            if (j < kept) {
                p = a.table[i * a.ld_table + j];
                if (p >= n && p < a.n_pages) p = a.dst[live_below(a.ws, before, p) - stay];
            }
            a.out[i * a.ld_out + j] = p;
        }
    }
}

dim3 rows_grid(int64_t n) { return dim3((unsigned)std::min<int64_t>(std::max<int64_t>(n, 1), 16384)); }

}  // namespace

int launch_kv_copy(const CopyArgs &a, hipStream_t stream) {
    int64_t chunks = 0;
    for (int i = 0; i < a.planes; ++i) chunks += copy_chunks(a.plane[i]);
    if (chunks > max_groups(kCopyThreads)) return QK_ERR_INVALID_ARG;
    const int64_t most = max_groups(kCopyThreads) / chunks;  // pairs of one launch
    for (int64_t i = 0; i < a.n; i += most) {
        CopyArgs p = a;
        p.n = std::min(a.n - i, most);
        p.src = a.src + i;
        p.dst = a.dst + i;
        const int st = launch(kv_copy_kernel, dim3((unsigned)(p.n * chunks)), dim3(kCopyThreads), stream, p, (int)chunks);
        if (st != QK_OK) return st;
    }
    return QK_OK;
}

int launch_kv_fork(const ForkArgs &a, hipStream_t stream) {
    const int64_t words = 2 * page_words(a.n_pages);
    int st = launch(clear_kernel, rows_grid((words + 255) / 256), dim3(256), stream, a.ws, words);
    if (st == QK_OK) st = launch(fork_mark_kernel, rows_grid(a.n_new), dim3(256), stream, a);
    if (st == QK_OK) st = launch(fork_plan_kernel, dim3(1), dim3(kPlanThreads), stream, a);
    if (st == QK_OK) st = launch(fork_write_kernel, rows_grid(a.n_new), dim3(256), stream, a);
    return st;
}

int launch_kv_compact(const CompactArgs &a, hipStream_t stream) {
    const int64_t words = page_words(a.n_pages);
    int st = launch(clear_kernel, rows_grid((words + 255) / 256), dim3(256), stream, a.ws, words);
    if (st == QK_OK) st = launch(compact_mark_kernel, rows_grid(a.n_rows), dim3(256), stream, a);
    if (st == QK_OK) st = launch(compact_plan_kernel, dim3(1), dim3(kPlanThreads), stream, a);
    if (st == QK_OK) st = launch(compact_write_kernel, rows_grid(a.n_rows), dim3(256), stream, a);
    return st;
}

}  // namespace qk
