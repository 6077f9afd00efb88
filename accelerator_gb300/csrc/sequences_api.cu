// sequences_api.cu -- the C ABI of what a batch of sequences needs around a cache
// (include/gemm.h): argument checks and dispatch.  Host code only.
#include <cstdint>

#include "api_checks.h"
#include "gemm.h"
#include "kernels.h"

namespace {

using namespace libgemm;

struct Span {
    const void* p;
    int64_t bytes;
    bool written;
};

}  // namespace

extern "C" {

int gemm_kv_plan(int32_t* page_table, int64_t table_width, const int32_t* lengths, const int32_t* counts,
                 const int32_t* free_pages, int64_t free_capacity, const int32_t* available, int32_t page_tokens,
                 int64_t tokens, int64_t sequences, int32_t* starts, int32_t* first, int32_t* new_lengths,
                 int32_t* heights, int32_t* left, int32_t* positions, int64_t* slots, struct CUstream_st* stream) {
    if (tokens < 0 || sequences < 0 || table_width < 0 || free_capacity < 0 || tokens > kIndexMax || sequences >= kIndexMax ||
        table_width > kIndexMax || free_capacity > kIndexMax || page_tokens < 1 || page_tokens > 1 << 20 ||
        (page_tokens & (page_tokens - 1)) != 0 || tokens / 256 + sequences + 1 > kIndexMax)
        return GEMM_ERR_INVALID_ARG;
    int log2 = 0;
    while (1 << log2 < page_tokens) ++log2;
    if (!starts || !heights || !left || !available || (sequences > 0 && (!lengths || !counts || !first || !new_lengths)) ||
        (tokens > 0 && (!positions || !slots)) || (free_capacity > 0 && !free_pages) ||
        (sequences > 0 && table_width > 0 && !page_table))
        return GEMM_ERR_INVALID_ARG;
    if (sequences > 0 && table_width > kElemMax / sequences) return GEMM_ERR_INVALID_ARG;
    enum { kTable, kLengths, kCounts, kFree, kAvailable, kStarts, kFirst, kAfter, kHeights, kLeft, kPositions, kSlots, kSpans };
    const Span spans[kSpans] = {{page_table, 4 * table_width * sequences, true}, {lengths, 4 * sequences, false},
                                {counts, 4 * sequences, false},                  {free_pages, 4 * free_capacity, false},
                                {available, 4, false},                           {starts, 4 * (sequences + 1), true},
                                {first, 4 * sequences, true},                    {new_lengths, 4 * sequences, true},
                                {heights, 4 * (sequences + 1), true},            {left, 4, true},
                                {positions, 4 * tokens, true},                   {slots, 8 * tokens, true}};
    for (int i = 0; i < kSpans; ++i)
        if (spans[i].bytes > 0 && !aligned(spans[i].p, i == kSlots ? 8 : 4)) return GEMM_ERR_MISALIGNED;
    for (int i = 0; i < kSpans; ++i)
        for (int j = 0; j < kSpans; ++j) {
            const Span &x = spans[i], &y = spans[j];
            const bool in_place = x.p == y.p && ((i == kAfter && j == kLengths) || (i == kLeft && j == kAvailable));
            if (i != j && x.written && !in_place && overlap(x.p, x.bytes, y.p, y.bytes)) return GEMM_ERR_INVALID_ARG;
        }
    int sms = 0;
    unsigned* err = nullptr;
    int rc = device_setup(&sms, &err);
    if (rc != GEMM_OK) return rc;
    const StepPlan plan{page_table, lengths, counts, free_pages, available, starts, first, new_lengths, heights, left, positions,
                        slots, table_width, free_capacity, tokens, sequences, log2};
    int launches = 0;
    if (launch_step_plan(plan, err, &launches, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) rc = GEMM_ERR_CUDA;
    for (int i = 0; i < launches; ++i) count_launch();
    return rc;
}

int gemm_rotary(const void* Q, int64_t q_row_stride, int64_t q_head_stride, void* Q_out, int64_t q_out_row_stride,
                int64_t q_out_head_stride, int32_t q_heads, const void* K, int64_t k_row_stride, int64_t k_head_stride,
                void* K_out, int64_t k_out_row_stride, int64_t k_out_head_stride, int32_t k_heads, int type, int64_t rows,
                int32_t head_dim, int32_t rotary_dim, int layout, const int32_t* positions, const uint64_t* turns,
                float magnitude, int inverse, struct CUstream_st* stream) {
    if (!type_ok(type) || rows < 0 || rows > kIndexMax || q_heads < 1 || q_heads > 32767 || k_heads < 0 || k_heads > 32767 ||
        head_dim < 2 || head_dim > 1024 || rotary_dim < 2 || rotary_dim > head_dim || rotary_dim % 2 != 0 ||
        (layout != GEMM_ROTARY_HALF && layout != GEMM_ROTARY_INTERLEAVED) || !(magnitude == magnitude))
        return GEMM_ERR_INVALID_ARG;
    if (rows == 0) return GEMM_OK;
    const int64_t es = type_size(type);
    const RotaryArgs a{{{{const_cast<void*>(Q), q_row_stride, q_head_stride}, {Q_out, q_out_row_stride, q_out_head_stride}, q_heads},
                        {{const_cast<void*>(K), k_row_stride, k_head_stride}, {K_out, k_out_row_stride, k_out_head_stride}, k_heads}},
                       rows, head_dim, rotary_dim, positions, turns, magnitude};
    if (!positions || !turns) return GEMM_ERR_INVALID_ARG;
    for (const RotaryRows& x : a.x) {
        if (x.heads == 0) continue;
        if (!x.in.p || !x.out.p || !strides_ok(rows, x.heads, x.in.row, x.in.head) || !strides_ok(rows, x.heads, x.out.row, x.out.head))
            return GEMM_ERR_INVALID_ARG;
    }
    for (const RotaryRows& x : a.x)
        if (x.heads > 0 && (!aligned(x.in.p, es) || !aligned(x.out.p, es))) return GEMM_ERR_MISALIGNED;
    if (!aligned(positions, 4) || !aligned(turns, 8)) return GEMM_ERR_MISALIGNED;
    auto apart = [&](const KvRows& p, int p_heads, const KvRows& q, int heads) {
        return rows_apart(p.p, p.row, p.head, p_heads, q.p, q.row, q.head, heads, rows, head_dim, es);
    };
    for (int i = 0; i < 2; ++i) {
        const RotaryRows &x = a.x[i], &y = a.x[1 - i];
        if (x.heads == 0) continue;
        const bool in_place = x.in.p == x.out.p && (rows == 1 || x.in.row == x.out.row) && (x.heads == 1 || x.in.head == x.out.head);
        const int64_t bytes = rows_span(rows, x.heads, head_dim, x.out.row, x.out.head, es);
        if (overlap_within(rows, x.heads, head_dim, x.out.row, x.out.head) || (!in_place && !apart(x.out, x.heads, x.in, x.heads)) ||
            (y.heads > 0 && (!apart(x.out, x.heads, y.in, y.heads) || !apart(x.out, x.heads, y.out, y.heads))) ||
            overlap(x.out.p, bytes, positions, 4 * rows) || overlap(x.out.p, bytes, turns, 4 * rotary_dim))
            return GEMM_ERR_INVALID_ARG;
    }
    int sms = 0;
    unsigned* err = nullptr;
    const int rc = device_setup(&sms, &err);
    if (rc != GEMM_OK) return rc;
    if (launch_rotary(a, static_cast<ElemType>(type), layout == GEMM_ROTARY_INTERLEAVED, inverse != 0, sms,
                      reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
        return GEMM_ERR_CUDA;
    count_launch();
    return GEMM_OK;
}

}  // extern "C"
