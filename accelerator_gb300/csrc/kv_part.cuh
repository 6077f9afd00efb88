// kv_part.cuh -- the units of the calls that write and read a paged cache.
#pragma once

#include "kernels.h"
#include "lowbit.cuh"

namespace libgemm {

// The part of a block of tokens that a unit of a launch is about.
struct Part {
    int64_t row;       // the batch row of the first token of the part
    int64_t page;
    int at;            // the block's first token in the page
    int begin, end;    // the part's tokens, counted from there
};

// Blocks are of B = 2^log2 tokens, a page or an equal part of one.  Sequence
// q's blocks are units floor(starts[q] / B) + 2q + j: T rows touch at most
// floor(T / B) + 2 of them, which is how far apart these are.
__device__ __forceinline__ bool find_part(const KvView& c, const KvBatch& b, int log2, int64_t u, unsigned* err, Part& part) {
    const bool report = threadIdx.x == 0 && blockIdx.y == 0;
    const Starts starts{b.starts, b.sequences, b.rows};
    const int B = 1 << log2;
    if (u == 0 && blockIdx.y == 0) starts.check(err);
    const int q = last_not_above(b.sequences, u, u / 2, [&](int i) { return (starts.at(i) >> log2) + 2 * (int64_t)i; });
    const int64_t row0 = starts.at(q), count = starts.at(q + 1) - row0, first = __ldg(b.at + q);
    if (!starts.good(q) || (count > 0 && (first < 0 || first + count > (b.width << c.page_log2)))) {
        if (report) atomicOr(err, kErrIndex);
        return false;
    }
    const int64_t blk = (first >> log2) + u - (row0 >> log2) - 2 * (int64_t)q, lo = blk << log2;
    // (a unit before the sequence's: where offsets descend the search may end there)
    if (count == 0 || blk < first >> log2 || lo >= first + count) return false;
    part.begin = (int)(first > lo ? first - lo : 0);
    part.end = (int)(first + count - lo < B ? first + count - lo : B);
    part.row = row0 + lo + part.begin - first;
    part.at = (int)(lo & ((1 << c.page_log2) - 1));
    part.page = __ldg(b.table + q * b.width + (lo >> c.page_log2));
    if (part.page < 0 || part.page >= c.pages) {
        if (report) atomicOr(err, kErrIndex);
        return false;
    }
    return true;
}

}  // namespace libgemm
