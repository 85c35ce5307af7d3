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
//
// What bounds them: a large copy its traffic (a list of 2000 pages of 64 KB of which 1800
// are copied, 236 MB read and written together, 47 us or 5.0 TB/s; 41 where the Infinity
// Cache holds a part of them from the call before), a small one its launch and two
// dependent loads (8 pages of 34 KB 2.5 us), a long list of few moves the workgroups that
// find nothing to do (100 moves in a list of 32768 65 us, in one of 100 3.5).  Tables are
// small and their work is a chain of passes that each wait for the one before
// (rows, bits, ranks, places): one workgroup's latency, 5.9 us for 4 rows of
// 63 pages, 13.1 for 64 rows of 256 (16384 entries through one CU); to pack, 7.1
// and 13.5 with the second launch that rewrites the tables.
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
constexpr int kCopyUnroll = 2;    // pieces of a thread

// Byte of piece `at` (bytes from the beginning) of a page.
__device__ __forceinline__ int64_t run_offset(const CopyPlane &p, int64_t at) {
    if (p.run == 0) return at;
    if (p.bytes <= INT32_MAX) {
        const uint32_t r = (uint32_t)at / p.run, o = r / p.inner;
        return (int64_t)o * p.outer_stride + (int64_t)(r - o * p.inner) * p.inner_stride + (uint32_t)at - r * p.run;
    }
    const int64_t r = at / p.run, o = r / p.inner;
    return o * p.outer_stride + (r - o * p.inner) * p.inner_stride + at - r * p.run;
}

constexpr int kCopyStep = kCopyThreads * kCopyUnroll;   // pieces of a workgroup

// STREAM: with stores that leave the caches alone (2000 pages of 64 KB 57 -> 43 us,
// 262 MB read and written together; no difference where the pages fit the caches).
template <typename PIECE, bool STREAM>
__device__ __forceinline__ void copy_chunk(const CopyPlane &p, int src, int dst, int64_t chunk) {
    PIECE x[kCopyUnroll];
    int64_t off[kCopyUnroll];
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u) {
        const int64_t at = (chunk * kCopyStep + u * kCopyThreads + threadIdx.x) * (int64_t)sizeof(PIECE);
        off[u] = at < p.bytes ? run_offset(p, at) : -1;
        if (off[u] >= 0) x[u] = *reinterpret_cast<const PIECE *>(p.base + src * p.page_stride + off[u]);
    }
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u) {
        PIECE *to = reinterpret_cast<PIECE *>(p.base + dst * p.page_stride + off[u]);
        if (off[u] < 0) continue;
        if (STREAM) __builtin_nontemporal_store(x[u], to);
        else *to = x[u];
    }
}

// Large pages: a workgroup takes one chunk of one plane of one pair.
template <bool STREAM>
__global__ __launch_bounds__(kCopyThreads) void kv_copy_kernel(const CopyArgs a) {
    const int64_t pair = a.first + blockIdx.x / (unsigned)a.chunks;
    int64_t c = blockIdx.x % (unsigned)a.chunks;
    const int src = a.src[pair], dst = a.dst[pair];
    if ((unsigned)src >= (unsigned)a.n_pages || (unsigned)dst >= (unsigned)a.n_pages || src == dst) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i >= a.planes) return;
        const CopyPlane &p = a.plane[i];
        const int64_t n = (p.pieces + kCopyStep - 1) / kCopyStep;
        if (c < n) {
            if (p.piece == 16) copy_chunk<u4_t, STREAM>(p, src, dst, c);
            else copy_chunk<uint32_t, STREAM>(p, src, dst, c);
            return;
        }
        c -= n;
    }
}

// Small pages: the pieces of all planes of all pairs in a row, a thread some of
// them (4000 pages of 2 KB 13 -> 4 us, in 8 bits 32 -> 5).
__global__ __launch_bounds__(kCopyThreads) void kv_copy_small_kernel(const CopyArgs a) {
    const uint32_t pieces = (uint32_t)a.pieces;
    const int64_t begin = (int64_t)blockIdx.x * kCopyStep;
    const int64_t pair0 = begin / pieces;
    const uint32_t rest = (uint32_t)(begin - pair0 * pieces);
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u) {
        const uint32_t at = rest + u * kCopyThreads + threadIdx.x;
        const uint32_t more = at / pieces;
        int64_t piece = at - more * pieces;
        const int64_t pair = a.first + pair0 + more;
        if (pair >= a.n) return;
        const int src = a.src[pair], dst = a.dst[pair];
        if ((unsigned)src >= (unsigned)a.n_pages || (unsigned)dst >= (unsigned)a.n_pages || src == dst) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i >= a.planes || piece < 0) break;
            const CopyPlane &p = a.plane[i];
            if (piece < p.pieces) {
                const int64_t off = run_offset(p, piece * p.piece);
                const uint8_t *from = p.base + src * p.page_stride + off;
                uint8_t *to = p.base + dst * p.page_stride + off;
                if (p.piece == 16) *reinterpret_cast<u4_t *>(to) = *reinterpret_cast<const u4_t *>(from);
                else *reinterpret_cast<uint32_t *>(to) = *reinterpret_cast<const uint32_t *>(from);
            }
            piece -= p.pieces;
        }
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

// Entry j of row i of the new table, `old` in the row that it is taken from (-1
// past what is taken); the row's requests are those from `rank` up to `next`.
__device__ __forceinline__ void fork_write(const ForkArgs &a, int i, int j, const Row &r, int old, int rank, int next, int found,
                                           const int *list) {
    // (a copied page is the one request that does not extend the row)
    const int copied = next - rank > r.want - min(r.kept, r.want) ? r.had / a.page_size : -1;
    const int request = j == copied ? rank : j >= r.kept && j < r.want ? rank + (copied >= 0) + j - r.kept : -1;
    int p = old;
    if (request >= 0) {
        p = request < found ? list[request] : -1;
        if (j == copied) {
            a.src[i] = p >= 0 ? old : -1;
            a.dst[i] = p;
        }
    }
    a.out[i * a.ld_out + j] = p;
    if (copied < 0 && j == 0) a.src[i] = a.dst[i] = -1;
}

__global__ __launch_bounds__(256) void fork_write_kernel(const ForkArgs a) {
    const int *list = reinterpret_cast<const int *>(a.ws + 2 * page_words(a.n_pages)), *first = list + a.n_pages;
    const int found = first[a.n_new + 1];
    for (int i = blockIdx.x; i < a.n_new; i += gridDim.x) {
        const Row r = fork_row(a, i);
        const int32_t *row = a.table + r.parent * a.ld_table;
        for (int j = threadIdx.x; j < a.out_pages; j += 256)
            fork_write(a, i, j, r, j < r.kept ? row[j] : -1, first[i], first[i + 1], found, list);
        if (a.out_pages == 0 && threadIdx.x == 0) a.src[i] = a.dst[i] = -1;
    }
}

// Tables and pools up to these sizes are planned by one workgroup, the bits in
// LDS: one launch instead of four.  In us with one / four, each row's last page
// copied: fork of 4 rows of 63 pages 5.7 / 11.5, 64 of 256 13 / 19, 1024 of 16 16 / 29,
// 1024 of 64 41 / 44, 256 of 256 38 / 33, 64 of 1024 37 / 26; each row grown in its place
// 64 of 256 11 / 14, 64 of 1024 33 / 18; packed 64 of 256 11 / 14, 64 of 1024 17 / 16.  So
// forks of few long rows are quicker in four launches from about 30000 entries on.
constexpr int kOneRows = 1024, kOneList = 4096;
constexpr int64_t kOnePages = 1 << 18, kOneEntries = 1 << 16;

// Threads side by side in a row: 2^shift, 16 at least.
__device__ __forceinline__ int row_shift(int pages) { return 32 - __clz((min(max(pages, 1), kPlanThreads) - 1) | 15); }

// Marks the pages that rows hold: threads side by side in a row, several rows'
// ids on their way at a time.  row(i) gives a row's ids and how many count.
template <typename ROW>
__device__ __forceinline__ void mark_rows(uint32_t *held, uint32_t *twice, int n_pages, int n, int pages, ROW row) {
    constexpr int U = 8;
    const int shift = row_shift(pages);
    const int step = kPlanThreads >> shift;
    for (int j0 = 0; j0 < pages; j0 += 1 << shift) {
        const int j = j0 + (threadIdx.x & ((1 << shift) - 1));
        for (int i0 = threadIdx.x >> shift; i0 < n; i0 += U * step) {
            int p[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * step;
                p[u] = -1;
                if (i < n) {
                    int kept;
                    const int32_t *ids = row(i, kept);
                    if (j < kept) p[u] = ids[j];
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if ((unsigned)p[u] >= (unsigned)n_pages) continue;
                const uint32_t bit = 1u << (p[u] & 31), was = atomicOr(&held[p[u] >> 5], bit);
                if (twice != nullptr && (was & bit)) atomicOr(&twice[p[u] >> 5], bit);
            }
        }
    }
}

// A new row: whose pages it takes over, how many, how many it has in all, and
// which of them is to be copied (-1: none).
struct __attribute__((aligned(16))) Taken { int parent, kept, want, copied; };

__global__ __launch_bounds__(kPlanThreads) void fork_one_kernel(const ForkArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint32_t lds[];
    __shared__ Taken taken[kOneRows];
    __shared__ int first[kOneRows], found_list[kOneList], sums[kPlanThreads / 64];
    const int words = (int)page_words(a.n_pages);
    uint32_t *held = lds, *twice = held + words;
    for (int w = threadIdx.x; w < 2 * words; w += kPlanThreads) held[w] = 0;
    Row mine{};
    if ((int)threadIdx.x < a.n_new) {
        mine = fork_row(a, threadIdx.x);
        taken[threadIdx.x] = Taken{mine.parent, mine.kept, mine.want, -1};
    }
    __syncthreads();
    mark_rows(held, twice, a.n_pages, a.n_new, min(a.in_pages, a.out_pages), [&](int i, int &kept) {
        const Taken t = taken[i];
        kept = t.kept;
        return a.table + t.parent * a.ld_table;
    });
    __syncthreads();
    // requests before each row
    int need = 0, asked;
    if ((int)threadIdx.x < a.n_new) {
        need = mine.want - min(mine.kept, mine.want);
        if (mine.has > mine.had && mine.had % a.page_size != 0) {
            const int last = mine.had / a.page_size;
            const int p = a.table[mine.parent * a.ld_table + last];
            if ((unsigned)p < (unsigned)a.n_pages && (twice[p >> 5] >> (p & 31) & 1)) {
                ++need;
                taken[threadIdx.x].copied = last;
            }
        }
    }
    const int before = block_scan(need, asked, sums);
    if ((int)threadIdx.x < a.n_new) first[threadIdx.x] = before;
    // the free pages, each thread some words in a row
    int *list = asked <= kOneList ? found_list : reinterpret_cast<int *>(a.ws);
    const int each = (words + kPlanThreads - 1) / kPlanThreads, w0 = min((int)threadIdx.x * each, words), w1 = min(w0 + each, words);
    auto free_in = [&](int w) { return ~held[w] & low_bits(min(32, a.n_pages - 32 * w)); };
    int count = 0, found;
    for (int w = w0; w < w1; ++w) count += __popc(free_in(w));
    int rank = block_scan(count, found, sums);
    for (int w = w0; w < w1 && rank < asked; ++w)
        for (uint32_t free = free_in(w); free != 0 && rank < asked; free &= free - 1) list[rank++] = 32 * w + __builtin_ctz(free);
    if (threadIdx.x == 0) *a.missing = max(0, asked - found);
    __syncthreads();
    // what rows take over, then what they asked for, a thread each
    constexpr int U = 8;   // entries of a thread on the way at a time
    const int shift = row_shift(a.out_pages), step = kPlanThreads >> shift;
    for (int j0 = 0; j0 < a.out_pages; j0 += 1 << shift) {
        const int j = j0 + (threadIdx.x & ((1 << shift) - 1));
        for (int i0 = threadIdx.x >> shift; i0 < a.n_new; i0 += U * step) {
            int p[U];
            bool mine[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * step;
                const Taken t = taken[min(i, a.n_new - 1)];
                mine[u] = i < a.n_new && j < a.out_pages && j != t.copied && (j < t.kept || j >= t.want);
                p[u] = mine[u] && j < t.kept ? a.table[t.parent * a.ld_table + j] : -1;
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (mine[u]) a.out[(i0 + u * step) * a.ld_out + j] = p[u];
        }
    }
    for (int q = threadIdx.x; q < asked; q += kPlanThreads) {
        int lo = 0, hi = a.n_new - 1;   // the last row whose requests begin at or before q
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first[mid] <= q) lo = mid;
            else hi = mid - 1;
        }
        const Taken t = taken[lo];
        const int at = q - first[lo], got = q < found ? list[q] : -1;
        int j = t.kept + at;
        if (t.copied >= 0) {
            j = at == 0 ? t.copied : j - 1;
            if (at == 0) {
                a.src[lo] = got >= 0 ? a.table[t.parent * a.ld_table + j] : -1;
                a.dst[lo] = got;
            }
        }
        a.out[lo * a.ld_out + j] = got;
    }
    if ((int)threadIdx.x < a.n_new && taken[threadIdx.x].copied < 0) a.src[threadIdx.x] = a.dst[threadIdx.x] = -1;
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

// The m-th free page (there is one): the last word with no more than m before it.
__device__ __forceinline__ int free_page(const uint32_t *held, const int *before, int words, int m) {
    int lo = 0, hi = words - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (32 * mid - before[mid] <= m) lo = mid;
        else hi = mid - 1;
    }
    uint32_t free = ~held[lo];
    for (int k = m - (32 * lo - before[lo]); k > 0; --k) free &= free - 1;
    return 32 * lo + __builtin_ctz(free);
}

// The live pages before each word, their number, and how many of them stay.
__device__ __forceinline__ void compact_plan(const CompactArgs &a, const uint32_t *held, int *before, int words, int (&sums)[kPlanThreads / 64]) {
    const int each = (words + kPlanThreads - 1) / kPlanThreads, w0 = min((int)threadIdx.x * each, words), w1 = min(w0 + each, words);
    int count = 0, n;
    for (int w = w0; w < w1; ++w) count += __popc(held[w]);
    int b = block_scan(count, n, sums);
    for (int w = w0; w < w1; ++w) {
        before[w] = b;
        b += __popc(held[w]);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        *a.live = n;
        before[words] = n;
        before[words + 1] = n < a.n_pages ? live_below(held, before, n) : n;
    }
}

__global__ __launch_bounds__(kPlanThreads) void compact_plan_kernel(const CompactArgs a) {
    __shared__ int sums[kPlanThreads / 64];
    const int words = (int)page_words(a.n_pages);
    compact_plan(a, a.ws, reinterpret_cast<int *>(a.ws + words), words, sums);
}

// Marking and plan of small tables and pools, the bits in LDS.
__global__ __launch_bounds__(kPlanThreads) void compact_one_kernel(const CompactArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint32_t lds[];
    __shared__ int kept[kOneRows], sums[kPlanThreads / 64];
    const int words = (int)page_words(a.n_pages);
    for (int w = threadIdx.x; w < words; w += kPlanThreads) lds[w] = 0;
    if ((int)threadIdx.x < a.n_rows) kept[threadIdx.x] = compact_kept(a, threadIdx.x);
    __syncthreads();
    mark_rows(lds, nullptr, a.n_pages, a.n_rows, a.max_pages, [&](int i, int &k) {
        k = kept[i];
        return a.table + i * a.ld_table;
    });
    __syncthreads();
    compact_plan(a, lds, reinterpret_cast<int *>(a.ws + words), words, sums);
    for (int w = threadIdx.x; w < words; w += kPlanThreads) a.ws[w] = lds[w];
}

// Which pages move where: the m-th live page from n on (n = the number of live
// pages) to the m-th free one below n; and the rows with the new ids.
__global__ __launch_bounds__(256) void compact_write_kernel(const CompactArgs a) {
    const int words = (int)page_words(a.n_pages);
    const uint32_t *held = a.ws;
    const int *before = reinterpret_cast<const int *>(a.ws + words);
    const int n = before[words], stay = before[words + 1];
    const int64_t all = (int64_t)gridDim.x * 256, at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    // page p, live and moved or free and moved to
    for (int64_t p = at; p < a.n_pages; p += all) {
        const int live = live_below(held, before, (int)p);
        const bool is = held[p >> 5] >> (p & 31) & 1;
        if (is && p >= n) a.src[live - stay] = (int)p;
        if (!is && p < n) a.dst[p - live] = (int)p;
    }
    for (int64_t m = n - stay + at; m < a.n_pages / 2; m += all) a.src[m] = a.dst[m] = -1;
    const int64_t entries = (int64_t)a.n_rows * a.max_pages;
    for (int64_t e = at; e < entries; e += all) {
        const uint32_t i = (uint32_t)e / (uint32_t)a.max_pages, j = (uint32_t)e - i * (uint32_t)a.max_pages;
        int p = -1;
        if ((int)j < compact_kept(a, (int)i)) {
            p = a.table[i * a.ld_table + j];
            if (p >= n && p < a.n_pages) p = free_page(held, before, words, live_below(held, before, p) - stay);
        }
        a.out[i * a.ld_out + j] = p;
    }
}

// A launch with more LDS than a kernel has without asking.
template <typename KERNEL, typename ARGS>
int launch_big(KERNEL kern, dim3 grid, dim3 block, size_t lds, hipStream_t stream, const ARGS &a) {
    if (lds > 16384 && hipFuncSetAttribute(reinterpret_cast<const void *>(kern), hipFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)lds) != hipSuccess)
        return QK_ERR_LAUNCH;
    return launch_lds(kern, grid, block, lds, stream, a);
}

dim3 rows_grid(int64_t n) { return dim3((unsigned)std::min<int64_t>(std::max<int64_t>(n, 1), 16384)); }

}  // namespace

int launch_kv_copy(const CopyArgs &args, hipStream_t stream) {
    CopyArgs a = args;
    int64_t bytes = 0, chunks = 0;
    a.pieces = 0;
    for (int i = 0; i < a.planes; ++i) {
        CopyPlane &p = a.plane[i];
        // 16 bytes where runs begin and end at multiples of them
        const uint64_t all = (uint64_t)(uintptr_t)p.base | (uint64_t)p.page_stride | (uint64_t)p.outer_stride |
                             (uint64_t)p.inner_stride | (uint64_t)p.bytes | p.run;
        p.piece = all % 16 == 0 ? 16 : 4;
        p.pieces = p.bytes / p.piece;
        a.pieces += p.pieces;
        chunks += (p.pieces + kCopyStep - 1) / kCopyStep;
        bytes += p.bytes;
    }
    if (chunks > max_groups(kCopyThreads)) return QK_ERR_INVALID_ARG;   // (a page of 2^36 bytes)
    a.chunks = (int)chunks;
    const bool small = a.plane[0].pieces < kCopyStep / 2, stream_out = a.n * (double)bytes >= 64e6;
    // pairs of one launch
    const int64_t most = small ? max_groups(kCopyThreads) * kCopyStep / a.pieces - 1 : max_groups(kCopyThreads) / chunks;
    for (int64_t i = 0; i < args.n; i += most) {
        a.first = i;
        a.n = std::min(args.n, i + most);
        const dim3 grid((unsigned)(small ? ((a.n - i) * a.pieces + kCopyStep - 1) / kCopyStep : (a.n - i) * chunks)), block(kCopyThreads);
        const int st = small        ? launch(kv_copy_small_kernel, grid, block, stream, a)
                       : stream_out ? launch(kv_copy_kernel<true>, grid, block, stream, a)
                                    : launch(kv_copy_kernel<false>, grid, block, stream, a);
        if (st != QK_OK) return st;
    }
    return QK_OK;
}

int launch_kv_fork(const ForkArgs &a, hipStream_t stream) {
    if (a.n_new <= kOneRows && a.n_pages <= kOnePages && (int64_t)a.n_new * std::max(a.in_pages, a.out_pages) <= kOneEntries)
        return launch_big(fork_one_kernel, dim3(1), dim3(kPlanThreads), 8 * (size_t)page_words(a.n_pages), stream, a);
    const int64_t words = 2 * page_words(a.n_pages);
    int st = launch(clear_kernel, rows_grid((words + 255) / 256), dim3(256), stream, a.ws, words);
    if (st == QK_OK) st = launch(fork_mark_kernel, rows_grid(a.n_new), dim3(256), stream, a);
    if (st == QK_OK) st = launch(fork_plan_kernel, dim3(1), dim3(kPlanThreads), stream, a);
    if (st == QK_OK) st = launch(fork_write_kernel, rows_grid(a.n_new), dim3(256), stream, a);
    return st;
}

int launch_kv_compact(const CompactArgs &a, hipStream_t stream) {
    const int64_t words = page_words(a.n_pages);
    int st;
    if (a.n_rows <= kOneRows && a.n_pages <= kOnePages && (int64_t)a.n_rows * a.max_pages <= kOneEntries) {
        st = launch_big(compact_one_kernel, dim3(1), dim3(kPlanThreads), 4 * (size_t)words, stream, a);
    } else {
        st = launch(clear_kernel, rows_grid((words + 255) / 256), dim3(256), stream, a.ws, words);
        if (st == QK_OK) st = launch(compact_mark_kernel, rows_grid(a.n_rows), dim3(256), stream, a);
        if (st == QK_OK) st = launch(compact_plan_kernel, dim3(1), dim3(kPlanThreads), stream, a);
    }
    if (st == QK_OK) st = launch(compact_write_kernel, rows_grid((std::max<int64_t>((int64_t)a.n_rows * a.max_pages, a.n_pages) + 255) / 256), dim3(256), stream, a);
    return st;
}

}  // namespace qk
