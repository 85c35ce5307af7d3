// kv_pages.h - launch descriptors of the calls on whole pages of a cache and
// on page tables (host and device).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qk {

// Elements of one page that are copied: `outer` times `inner` runs of `run`
// bytes (runs that lie back to back joined into one).
struct CopyPlane {
    uint8_t *base;
    int64_t page_stride, outer_stride, inner_stride;   // bytes
    uint32_t inner, run;                               // runs per outer step; bytes of a run (0: one run)
    int64_t bytes;                                     // of one page
    int64_t pieces;                                    // of `piece` bytes in a page
    int piece;
};

struct CopyArgs {
    CopyPlane plane[4];     // keys, values, and the scales of 8 bits
    int planes;
    const int32_t *src, *dst;
    int64_t first, n;       // pairs first .. n - 1
    int64_t pieces;         // of a page's planes together
    int chunks;             // workgroups of a pair, planes apart
    int n_pages;
};

struct ForkArgs {
    const int32_t *table, *lens, *parent, *new_lens;
    int32_t *out, *src, *dst, *missing;
    int64_t ld_table, ld_out;
    int n_rows, n_new, in_pages, out_pages, page_size, n_pages;
    uint32_t *ws;
};

struct CompactArgs {
    const int32_t *table, *lens;
    int32_t *out, *src, *dst, *live;
    int64_t ld_table, ld_out;
    int n_rows, max_pages, page_size, n_pages;
    uint32_t *ws;
};

// 32-bit words of scratch: two bits per page, the free pages found (or the
// live pages before each word), and the requests before each row.
constexpr int64_t page_words(int64_t n_pages) { return (n_pages + 31) / 32; }
constexpr int64_t pages_ws_words(int64_t n_rows, int64_t n_pages) {
    return 2 * page_words(n_pages) + n_pages + n_rows + 4;
}

int launch_kv_copy(const CopyArgs &a, hipStream_t stream);
int launch_kv_fork(const ForkArgs &a, hipStream_t stream);
int launch_kv_compact(const CompactArgs &a, hipStream_t stream);

}  // namespace qk
