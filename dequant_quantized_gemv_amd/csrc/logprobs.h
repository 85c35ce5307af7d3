// logprobs.h - launch descriptor of the log probabilities (host and device).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

namespace qk {

constexpr int kLogpThreads = 1024;
constexpr int kLogpTop = 64;      // best alternatives of a row, at most
constexpr int kLogpMost = 32;     // logits of a thread
constexpr int kLogpLeast = 8;
constexpr uint32_t kLogpList = 512;   // candidates for the best

struct LogpArgs {
    const void *x;
    const int32_t *ids;
    float *lp, *entropy, *best;
    int32_t *best_ids;
    int64_t ldx, ld_ids, ld_lp, ld_best_ids, ld_best;
    int64_t n;
    int vocab, n_ids, top, parts;
    float scale, scale2;   // the second times log2(e)
    float *stat;        // 4 per (row, part)
    uint64_t *list;     // `top` per (row, part)
};

// A row goes to workgroups of `threads` in parts of threads * each logits.
struct LogpSplit {
    int threads, each;
    int64_t part() const { return (int64_t)threads * each; }
    int64_t parts(int64_t vocab) const { return (vocab - 1) / part() + 1; }
};

// A part is as large as a workgroup holds (1024 lanes of 32), and no larger than a row
// needs: smaller ones for few long rows gain nothing (1 x 131072 with 20 best 12.9 us in
// 16 parts, 13.4 in 4; 64 of them 20.6 in either) and cost a join where a row would fit
// (64 x 32000 15.7 us in 8 parts, 10.6 in one).  Rows of one wave's or four waves'
// logits get no more waves (4096 x 1000 12 us, with 1024 lanes a row 112), but where
// there are too few of them for the card.
inline LogpSplit logp_split(int64_t n, int64_t vocab, int64_t cus) {
    if (vocab <= 64 * kLogpMost) return {64, kLogpMost};
    if (vocab <= 256 * kLogpMost && n >= 2 * cus) return {256, kLogpMost};
    LogpSplit s{kLogpThreads, kLogpMost};
    while (s.each > kLogpLeast && s.part() / 2 >= vocab) s.each /= 2;
    return s;
}

// Parts in scratch (of rows that have more than one).
inline int64_t logp_parts(int64_t n, int64_t vocab) {
    const int64_t parts = LogpSplit{kLogpThreads, kLogpMost}.parts(vocab);
    return parts > 1 ? n * parts : 0;
}

int launch_token_logprobs(const LogpArgs &a, bool f16, const LogpSplit &split, hipStream_t stream);

}  // namespace qk
