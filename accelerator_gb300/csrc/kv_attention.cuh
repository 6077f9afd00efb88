// kv_attention.cuh -- what the two attention kernels (few query rows and many)
// share: the arguments, the rows and tokens of a tile, and constants.
#pragma once

#include "kernels.h"
#include "lowbit.cuh"

namespace libgemm {

constexpr float kNegInf = -INFINITY, kLowest = -3.402823466e38f;
// Weights (with their page's value scale) enter the second product as binary16
// times 2^15 relative to the row's largest, under 2^16: the maximum that they are
// relative to may lag behind by this much (in log2).  A largest of less than
// 2^-110 counts as that.
constexpr float kPScale = 32768.0f, kLag = 0.9f, kMostP = 61147.0f /* 2^(15 + kLag) */, kLeast = 7.7037198e-34f;

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

struct AttnArgs {
    KvView c;
    KvRows Q, O;
    KvBatch b;
    int q_heads;
    unsigned share;              // query heads that read one cache head; rows * share fits 31 bits
    int gap;                     // a tile's rows less their greatest common divisor with share
    float scale_log2;            // scale * log2(e)
    int causal;
    int window;
    int splits;                  // CTAs that share a tile's tokens: a cluster, or with `partial` any number
    bool q_vec;                  // Q in 16-byte loads
    int64_t partial_bytes;
    float* partial;              // [unit][head][split] x (rows x dim sums, then rows x (max, sum))
    unsigned* err;
};

// The tile of a unit: its sequence and rows, and the tokens that it sees
// (token numbers fit 32 bits, as the lengths do).
struct Tile {
    int seq;
    int row0;                    // first of the sequence's rows
    int r0, nrows;               // first row (query, head pair) of the tile; rows of the sequence
    int len, p0;                 // cached tokens; position of query 0
    int tok0;                    // first token, a multiple of the step
    int lo, hi;                  // the tokens that any row sees: lo .. hi - 1
    int steps, per, active;      // steps in all, per split, splits that have any

    // Row r sees the tokens row_lo(r) .. row_hi(r) - 1; both grow with r.
    __device__ __forceinline__ int row_hi(const AttnArgs& a, int r) const {
        const int p = p0 + (int)((unsigned)r / a.share);
        if (p < 0) return 0;
        return a.causal ? p + 1 : len;
    }
    __device__ __forceinline__ int row_lo(const AttnArgs& a, int r) const {
        const int p = p0 + (int)((unsigned)r / a.share);
        return a.window > 0 && p >= a.window ? p - a.window + 1 : 0;
    }
    // Whether the page of token `tok` holds a token that any row sees: of a step
    // that begins before the window or ends past the last token, not all do, and
    // the table need not name those that do not.
    __device__ __forceinline__ bool page_seen(int tok, int page_log2) const {
        return tok < hi && tok >> page_log2 >= lo >> page_log2;
    }
    // `check` for one CTA of a unit: it reports what is out of range.
    __device__ __forceinline__ bool find(const AttnArgs& a, int u, int rows, int step, bool check) {
        const Starts starts{a.b.starts, a.b.sequences, a.b.rows};
        if (u == 0 && check) starts.check(a.err);
        // Sequence q's tiles are units unit_of(q) + j: its rows are a multiple of
        // share, so that they need at most (rows + gap) / tile tiles.
        auto unit_of = [&](int64_t start, int i) { return (int)((start * a.share + (int64_t)i * a.gap) / rows); };
        seq = last_not_above(a.b.sequences, u, u, [&](int i) { return unit_of(starts.at(i), i); });
        row0 = (int)starts.at(seq);
        const int count = (int)starts.at(seq + 1) - row0, length = __ldg(a.b.at + seq);
        if (!starts.good(seq)) {
            if (check && threadIdx.x == 0) atomicOr(a.err, kErrIndex);
            return false;
        }
        nrows = count * (int)a.share;
        r0 = (u - unit_of(row0, seq)) * rows;
        if (r0 < 0 || r0 >= nrows) return false;
        len = length;
        if (length < 0 || length > (a.b.width << a.c.page_log2)) {
            if (check && threadIdx.x == 0) atomicOr(a.err, kErrIndex);
            len = 0;
        }
        p0 = len - count;
        hi = row_hi(a, min(r0 + rows, nrows) - 1);
        lo = row_lo(a, r0);
        tok0 = lo / step * step;
        steps = hi > tok0 ? (hi - tok0 + step - 1) / step : 0;
        per = max(1, (steps + a.splits - 1) / a.splits);
        active = max(1, (steps + per - 1) / per);
        return true;
    }
};

// Where a row's results go.
template <typename T>
__device__ __forceinline__ T* out_row(const AttnArgs& a, const Tile& tile, int h, unsigned r) {
    return static_cast<T*>(a.O.p) + (int64_t)(tile.row0 + r / a.share) * a.O.row + (int64_t)(h * a.share + r % a.share) * a.O.head;
}

// Many query rows (kv_prompt.cu): tiles of plan.rows = 256, tokens in steps of 128.
cudaError_t kv_prompt_setup();
cudaError_t launch_kv_prompt(const AttnArgs& a, ElemType type, const KvPlan& plan, cudaStream_t stream);

}  // namespace libgemm
