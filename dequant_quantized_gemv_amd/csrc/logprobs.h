// logprobs.h - launch descriptor of the log probabilities (host and device).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

namespace qk {

constexpr int kLogpThreads = 512;
constexpr int kLogpMost = 64;     // logits of a thread, at most; and best alternatives of a row
constexpr int kLogpLeast = 8;

struct LogpArgs {
    const void *x;
    const int32_t *ids;
    float *lp, *entropy, *best;
    int32_t *best_ids;
    int64_t ldx, ld_ids, ld_lp, ld_best_ids, ld_best;
    int64_t n;
    int vocab, n_ids, top, parts;
    float scale;
    float *stat;        // 4 per (row, part)
    uint64_t *list;     // `top` per (row, part)
};

// A row goes to workgroups in parts of kLogpThreads times `each` logits: parts
// as large as leaves two workgroups for every CU, and no larger than a row.
inline int logp_each(int64_t n, int64_t vocab, int64_t cus) {
    int each = kLogpMost;
    while (each > kLogpLeast && ((int64_t)kLogpThreads * each / 2 >= vocab ||
                                 n * ((vocab - 1) / (kLogpThreads * each) + 1) < 2 * cus))
        each /= 2;
    return each;
}
inline int64_t logp_parts(int64_t vocab, int each) { return (vocab - 1) / (kLogpThreads * each) + 1; }

// Parts in scratch of any call of up to n rows of up to vocab logits: more than
// the largest parts would give are only made while there are fewer than
// 2 * cus of twice the size.
inline int64_t logp_parts_bound(int64_t n, int64_t vocab, int64_t cus) {
    const int64_t most = logp_parts(vocab, kLogpLeast);
    if (most == 1) return 0;
    return std::min(n * most, std::max(4 * cus, n * logp_parts(vocab, kLogpMost)));
}

int launch_token_logprobs(const LogpArgs &a, bool f16, int each, hipStream_t stream);

}  // namespace qk
