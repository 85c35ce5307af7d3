// attn.h - launch descriptors of the paged key-value cache (host and device):
// the store of new rows and the attention of one new token per sequence.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qk {

constexpr int kAttnTile = 32;      // tokens a wave takes at a time
constexpr int kAttnWaves = 4;      // waves per workgroup
constexpr int kAttnHeads = 16;     // query heads of one key-value head per workgroup

struct AttnArgs {
    const uint8_t *k, *v;          // pools
    const float *ks, *vs;          // scales (8-bit pools)
    const float *q;
    const int32_t *table;
    const int32_t *lens;
    void *y;
    float *part;                   // partial results, nchunks per (sequence, head); see attn_part_floats
    int64_t page_stride, head_stride, slot_stride;   // bytes of k and v
    int64_t sc_page, sc_head, sc_slot;               // elements of ks and vs
    int64_t q_seq, q_head, y_seq, y_head;            // elements
    int64_t ld_table;
    int n_seqs, n_heads, n_kv, group, head_tiles;
    int n_pages, page_size;
    uint32_t page_magic, page_shift;                 // t / page_size == t * page_magic >> page_shift, t < 2^30
    int max_len, window, sinks;
    int chunk_tiles, nchunks;
    float qscale;                  // softmax scale * log2(e)
    int out_f16;
};

// The attention of sequences of which groups share their first tokens: group g
// is sequences starts[g] .. starts[g + 1] - 1, shared[g] tokens in the pages of
// its first sequence.  A (sequence, head) has `slots` partial results, first
// those of the shared tokens' chunks, then those of its own (nchunks).
struct SharedArgs : AttnArgs {
    const int32_t *starts, *shared;
    int n_groups, max_shared, max_own;
    int prefix_tiles, prefix_chunks, slots;   // tiles of a chunk of shared tokens; chunks
    int row_tiles, row_waves;                 // tiles of query rows, at most; waves with rows of their own in each
    int seq0, group0;                         // first sequence, first eight of workgroups of this launch
    int own_blocks, own_items;                // workgroups of sequences' own tokens in it, chunks of those
    int own_waves;                            // waves of such a chunk, 4 or 1
};

// One partial result: the running maximum and sum, then head_dim outputs.
constexpr int64_t attn_part_floats(int head_dim) { return head_dim + 4; }

// The tokens a query sees, as 32-token tiles: with a window that begins past
// the first tokens kept visible, `ns` tiles of those and then the tiles from
// `start`; otherwise the tiles from `start` alone.
struct AttnSpan {
    int len, ws;    // tokens; first token of the window
    int start, ns, tiles;
};

__host__ __device__ inline AttnSpan attn_span(int len, int window, int sinks) {
    AttnSpan s;
    s.len = len;
    s.ws = window > 0 && len > window ? len - window : 0;
    const int ws32 = s.ws & ~(kAttnTile - 1);
    const bool apart = sinks < ws32;
    s.start = apart ? ws32 : 0;
    s.ns = apart ? (sinks + kAttnTile - 1) / kAttnTile : 0;
    s.tiles = s.ns + (len - s.start + kAttnTile - 1) / kAttnTile;
    return s;
}

// A sequence's own tokens behind `shared`.
__host__ __device__ inline AttnSpan own_span(int len, int shared) {
    const int start = shared & ~(kAttnTile - 1);
    return AttnSpan{len, shared, start, 0, (len - start + kAttnTile - 1) / kAttnTile};
}

// Tokens of a tile of the shared ones (as many bytes on their way with small
// heads), and query rows of one: `row_waves` (4, 2, or with tiles of 128 tokens 1)
// of a workgroup's waves have rows of their own.
constexpr int prefix_tokens(int head_dim) { return head_dim <= 64 ? 128 : 64; }
constexpr int prefix_rows(int row_waves) { return 32 * row_waves; }

struct StoreArgs {
    uint8_t *kc, *vc;
    float *ks, *vs;
    const float *k, *v;
    const int32_t *table, *seq, *pos;
    int64_t page_stride, head_stride, slot_stride;   // elements of kc and vc
    int64_t sc_page, sc_head, sc_slot;
    int64_t k_tok, k_head, v_tok, v_head;
    int64_t ld_table;
    int64_t tokens;
    int n_seqs, max_pages, n_pages, page_size, n_kv, head_dim;
};

template <bool I8> int attn_decode_run(const AttnArgs &a, int head_dim, bool tiled, hipStream_t stream);
template <bool I8> int attn_shared_run(const SharedArgs &a, int head_dim, bool tiled, hipStream_t stream);

}  // namespace qk
