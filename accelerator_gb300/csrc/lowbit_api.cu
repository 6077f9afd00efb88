// lowbit_api.cu -- the C ABI of the operators on operands held in few bits
// (include/gemm.h): argument checks and dispatch.  Host code only.
#include <cstdint>

#include "gemm.h"
#include "kernels.h"

namespace {

using namespace libgemm;

constexpr int64_t kIndexMax = 0x7FFFFFFF;          // sizes held in 32 bits, grids
constexpr int64_t kElemMax = INT64_MAX / 64;

bool type_ok(int type) { return type == GEMM_TYPE_F32 || type == GEMM_TYPE_BF16 || type == GEMM_TYPE_F16; }
int64_t type_size(int type) { return type == GEMM_TYPE_F32 ? 4 : 2; }
bool aligned(const void* p, int64_t to) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(to - 1)) == 0; }

bool overlap(const void* a, int64_t abytes, const void* b, int64_t bbytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return abytes > 0 && bbytes > 0 && x < y + (uint64_t)bbytes && y < x + (uint64_t)abytes;
}

// Bytes spanned by rows x cols elements of row stride ld.
int64_t span(int64_t rows, int64_t cols, int64_t ld, int64_t es) {
    return rows > 0 && cols > 0 ? ((rows - 1) * ld + cols) * es : 0;
}

int w4_shape(int64_t K, int64_t N, int group, int64_t* codes, int64_t* scales) {
    if (K < 0 || N < 0 || K > kIndexMax - 255 || N > kIndexMax - 255) return GEMM_ERR_INVALID_ARG;
    if (group != 32 && group != 64 && group != 128) return GEMM_ERR_INVALID_ARG;
    const int64_t nb = (N + 15) / 16, kb = (K + 63) / 64, groups = (K + group - 1) / group;
    if (((K + 127) / 128) * ((N + 31) / 32) > kIndexMax) return GEMM_ERR_INVALID_ARG;
    *codes = nb * kb * 512;
    *scales = nb * groups * 32;
    return GEMM_OK;
}

// A dense-in-a-row K x N matrix in B with its codes and scales: either
// direction of the conversion.
int w4_convert(const void* B, int64_t ldb, int type, int64_t K, int64_t N, int group,
               const void* codes, const void* scales, bool quantize, cudaStream_t stream) {
    int64_t cb = 0, sb = 0;
    const int shape = w4_shape(K, N, group, &cb, &sb);
    if (shape != GEMM_OK) return shape;
    if (!type_ok(type) || ldb < N) return GEMM_ERR_INVALID_ARG;
    if (K == 0 || N == 0) return GEMM_OK;
    if (ldb > kElemMax / K || !B || !codes || !scales) return GEMM_ERR_INVALID_ARG;
    const int64_t es = type_size(type);
    if (!aligned(B, es) || !aligned(codes, 16) || !aligned(scales, 16)) return GEMM_ERR_MISALIGNED;
    const int64_t bytes = span(K, N, ldb, es);
    if (overlap(B, bytes, codes, cb) || overlap(B, bytes, scales, sb) || overlap(codes, cb, scales, sb))
        return GEMM_ERR_INVALID_ARG;
    int sms = 0;
    unsigned* err = nullptr;
    const int rc = device_setup(&sms, &err);
    if (rc != GEMM_OK) return rc;
    const ElemType t = static_cast<ElemType>(type);
    const cudaError_t e =
        quantize ? launch_w4_quantize(B, ldb, t, K, N, group, const_cast<void*>(codes),
                                      const_cast<void*>(scales), stream)
                 : launch_w4_dequantize(codes, scales, K, N, group, const_cast<void*>(B), ldb, t, stream);
    if (e != cudaSuccess) return GEMM_ERR_CUDA;
    count_launch();
    return GEMM_OK;
}

// Checks what the calls on a cache share.
int kv_view(const gemm_kv_cache* c, const int32_t* table, int64_t width, const int32_t* starts,
            const int32_t* at, int64_t tokens, int64_t sequences, KvView* view, KvBatch* batch) {
    if (!c || tokens < 0 || sequences < 0 || width < 0 || tokens > kIndexMax || sequences > kIndexMax ||
        width > kIndexMax)
        return GEMM_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128) return GEMM_ERR_INVALID_ARG;
    int log2 = -1;
    for (int i = 4; i <= 7; ++i)
        if (c->page_tokens == 1 << i) log2 = i;
    if (log2 < 0 || c->heads < 1 || c->heads > 32767 || c->pages < 0 || c->pages > kIndexMax)
        return GEMM_ERR_INVALID_ARG;
    if (width > (kIndexMax - 1023) >> log2) return GEMM_ERR_INVALID_ARG;   // positions and the steps past them fit 32 bits
    if (tokens == 0) return GEMM_OK;
    if (sequences == 0) return GEMM_ERR_INVALID_ARG;
    if (!starts || !at || (width > 0 && !table)) return GEMM_ERR_INVALID_ARG;
    if (c->pages > 0 && (!c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales)) return GEMM_ERR_INVALID_ARG;
    if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 4) ||
        !aligned(c->v_scales, 4) || !aligned(table, 4) || !aligned(starts, 4) || !aligned(at, 4))
        return GEMM_ERR_MISALIGNED;
    *view = KvView{static_cast<uint8_t*>(c->k_codes), static_cast<uint8_t*>(c->v_codes), c->k_scales,
                   c->v_scales, c->pages, c->heads, log2, c->head_dim};
    *batch = KvBatch{table, starts, at, width, tokens, (int)sequences};
    return GEMM_OK;
}

bool strides_ok(int64_t rows, int64_t heads, int64_t row, int64_t head) {
    return row >= 0 && head >= 0 && row <= kElemMax / 4 / (rows > 0 ? rows : 1) && head <= kElemMax / 4 / heads;
}

int64_t rows_span(int64_t rows, int64_t heads, int64_t dim, int64_t row, int64_t head, int64_t es) {
    return rows > 0 ? ((rows - 1) * row + (heads - 1) * head + dim) * es : 0;
}

// Whether two elements of rows x heads x dim with these strides are one: a
// result that many threads write has to have a place for each.
bool overlap_within(int64_t rows, int64_t heads, int64_t dim, int64_t row, int64_t head) {
    if ((rows > 1 && row < dim) || (heads > 1 && head < dim)) return true;
    if (rows <= 1 || heads <= 1 || row >= (heads - 1) * head + dim || head >= (rows - 1) * row + dim) return false;
    for (int64_t h = 1; h < heads; ++h) {   // neither lies inside the other: h heads on as far as r rows on, or nearly?
        const int64_t below = h * head / row;
        for (int64_t r = below > 0 ? below : 1; r <= below + 1 && r < rows; ++r)
            if (r * row - h * head < dim && h * head - r * row < dim) return true;
    }
    return false;
}

bool overlaps_cache(const KvView& v, const void* p, int64_t bytes) {
    const int64_t codes = v.pages * v.heads * ((int64_t)v.dim << v.page_log2), scales = v.pages * v.heads * 4;
    return overlap(p, bytes, v.k, codes) || overlap(p, bytes, v.v, codes) || overlap(p, bytes, v.ks, scales) ||
           overlap(p, bytes, v.vs, scales);
}

}  // namespace

extern "C" {

int gemm_w4_sizes(int64_t K, int64_t N, int group, int64_t* code_bytes, int64_t* scale_bytes) {
    if (!code_bytes || !scale_bytes) return GEMM_ERR_INVALID_ARG;
    return w4_shape(K, N, group, code_bytes, scale_bytes);
}

int gemm_w4_quantize(const void* B, int64_t ldb, int type, int64_t K, int64_t N, int group,
                     void* codes, void* scales, struct CUstream_st* stream) {
    return w4_convert(B, ldb, type, K, N, group, codes, scales, true, reinterpret_cast<cudaStream_t>(stream));
}

int gemm_w4_dequantize(const void* codes, const void* scales, int64_t K, int64_t N, int group,
                       void* B, int64_t ldb, int type, struct CUstream_st* stream) {
    return w4_convert(B, ldb, type, K, N, group, codes, scales, false, reinterpret_cast<cudaStream_t>(stream));
}

int gemm_w4(const void* X, int64_t ldx, int x_type, const void* codes, const void* scales, void* C,
            int64_t ldc, int c_type, int64_t M, int64_t K, int64_t N, int group,
            struct CUstream_st* stream_) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    int64_t cb = 0, sb = 0;
    const int shape = w4_shape(K, N, group, &cb, &sb);
    if (shape != GEMM_OK) return shape;
    if (M < 0 || M > kIndexMax || ldx < K || ldc < N) return GEMM_ERR_INVALID_ARG;
    if ((x_type != GEMM_TYPE_BF16 && x_type != GEMM_TYPE_F16) || (c_type != GEMM_TYPE_F32 && c_type != x_type))
        return GEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return GEMM_OK;
    if (ldx > kElemMax / M || ldc > kElemMax / M || ((N + 31) / 32) * ((M + 7) / 8) > kIndexMax / 8)
        return GEMM_ERR_INVALID_ARG;
    if (!C || (K > 0 && (!X || !codes || !scales))) return GEMM_ERR_INVALID_ARG;
    const int64_t ces = type_size(c_type);
    if (!aligned(X, 2) || !aligned(C, ces) || !aligned(codes, 16) || !aligned(scales, 16)) return GEMM_ERR_MISALIGNED;
    const int64_t c_bytes = span(M, N, ldc, ces);
    if (overlap(C, c_bytes, X, span(M, K, ldx, 2)) || overlap(C, c_bytes, codes, cb) || overlap(C, c_bytes, scales, sb))
        return GEMM_ERR_INVALID_ARG;
    int sms = 0;
    unsigned* err = nullptr;
    const int rc = device_setup(&sms, &err);
    if (rc != GEMM_OK) return rc;
    if (launch_w4_gemm(X, ldx, static_cast<ElemType>(x_type), codes, scales, C, ldc,
                       static_cast<ElemType>(c_type), M, K, N, group, sms, stream) != cudaSuccess)
        return GEMM_ERR_CUDA;
    count_launch();
    return GEMM_OK;
}

int gemm_kv_append(const gemm_kv_cache* cache, const void* K, int64_t k_row_stride,
                   int64_t k_head_stride, const void* V, int64_t v_row_stride,
                   int64_t v_head_stride, int type, const int32_t* page_table, int64_t table_width,
                   const int32_t* starts, const int32_t* first, int64_t tokens, int64_t sequences,
                   struct CUstream_st* stream) {
    KvView v{};
    KvBatch b{};
    int rc = kv_view(cache, page_table, table_width, starts, first, tokens, sequences, &v, &b);
    if (rc != GEMM_OK) return rc;
    if (!type_ok(type)) return GEMM_ERR_INVALID_ARG;
    if (tokens == 0) return GEMM_OK;
    if (!K || !V || !strides_ok(tokens, v.heads, k_row_stride, k_head_stride) ||
        !strides_ok(tokens, v.heads, v_row_stride, v_head_stride))
        return GEMM_ERR_INVALID_ARG;
    const int64_t es = type_size(type);
    if (!aligned(K, es) || !aligned(V, es)) return GEMM_ERR_MISALIGNED;
    if (overlaps_cache(v, K, rows_span(tokens, v.heads, v.dim, k_row_stride, k_head_stride, es)) ||
        overlaps_cache(v, V, rows_span(tokens, v.heads, v.dim, v_row_stride, v_head_stride, es)))
        return GEMM_ERR_INVALID_ARG;
    if ((tokens >> v.page_log2) + 2 * sequences > kIndexMax) return GEMM_ERR_INVALID_ARG;
    int sms = 0;
    unsigned* err = nullptr;
    rc = device_setup(&sms, &err);
    if (rc != GEMM_OK) return rc;
    if (launch_kv_append(v, KvRows{const_cast<void*>(K), k_row_stride, k_head_stride},
                         KvRows{const_cast<void*>(V), v_row_stride, v_head_stride},
                         static_cast<ElemType>(type), b, err, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
        return GEMM_ERR_CUDA;
    count_launch();
    return GEMM_OK;
}

int gemm_kv_read(const gemm_kv_cache* cache, void* K, void* V, int type, const int32_t* page_table,
                 int64_t table_width, const int32_t* starts, const int32_t* first, int64_t tokens,
                 int64_t sequences, struct CUstream_st* stream) {
    KvView v{};
    KvBatch b{};
    int rc = kv_view(cache, page_table, table_width, starts, first, tokens, sequences, &v, &b);
    if (rc != GEMM_OK) return rc;
    if (!type_ok(type)) return GEMM_ERR_INVALID_ARG;
    if (tokens == 0) return GEMM_OK;
    if (!K || !V) return GEMM_ERR_INVALID_ARG;
    if (!aligned(K, 16) || !aligned(V, 16)) return GEMM_ERR_MISALIGNED;
    const int64_t bytes = tokens * v.heads * v.dim * type_size(type);
    if (overlaps_cache(v, K, bytes) || overlaps_cache(v, V, bytes) || overlap(K, bytes, V, bytes))
        return GEMM_ERR_INVALID_ARG;
    if ((tokens >> v.page_log2) + 2 * sequences > kIndexMax) return GEMM_ERR_INVALID_ARG;
    int sms = 0;
    unsigned* err = nullptr;
    rc = device_setup(&sms, &err);
    if (rc != GEMM_OK) return rc;
    if (launch_kv_read(v, K, V, static_cast<ElemType>(type), b, err, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
        return GEMM_ERR_CUDA;
    count_launch();
    return GEMM_OK;
}

int gemm_kv_attention(const gemm_kv_cache* cache, const void* Q, int64_t q_row_stride,
                      int64_t q_head_stride, void* O, int64_t o_row_stride, int64_t o_head_stride,
                      int type, int32_t q_heads, float scale, int causal, int64_t window,
                      const int32_t* page_table, int64_t table_width, const int32_t* starts,
                      const int32_t* lengths, int64_t tokens, int64_t sequences,
                      struct CUstream_st* stream_) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    KvView v{};
    KvBatch b{};
    int rc = kv_view(cache, page_table, table_width, starts, lengths, tokens, sequences, &v, &b);
    if (rc != GEMM_OK) return rc;
    if ((type != GEMM_TYPE_BF16 && type != GEMM_TYPE_F16) || q_heads < 1 || q_heads % cache->heads != 0 ||
        window < 0 || (window > 0 && !causal) || !(scale == scale))
        return GEMM_ERR_INVALID_ARG;
    if (tokens == 0) return GEMM_OK;
    if (!Q || !O || !strides_ok(tokens, q_heads, q_row_stride, q_head_stride) ||
        !strides_ok(tokens, q_heads, o_row_stride, o_head_stride))
        return GEMM_ERR_INVALID_ARG;
    if (!aligned(Q, 2) || !aligned(O, 2)) return GEMM_ERR_MISALIGNED;
    const int64_t q_bytes = rows_span(tokens, q_heads, v.dim, q_row_stride, q_head_stride, 2);
    const int64_t o_bytes = rows_span(tokens, q_heads, v.dim, o_row_stride, o_head_stride, 2);
    if (overlap(Q, q_bytes, O, o_bytes) || overlaps_cache(v, O, o_bytes) ||
        overlap_within(tokens, q_heads, v.dim, o_row_stride, o_head_stride))
        return GEMM_ERR_INVALID_ARG;
    if (tokens * (q_heads / v.heads) > kIndexMax - 16 || tokens * (q_heads / v.heads) / 8 + sequences > kIndexMax / 8 / v.heads)
        return GEMM_ERR_INVALID_ARG;
    int sms = 0;
    unsigned* err = nullptr;
    rc = device_setup(&sms, &err);
    if (rc != GEMM_OK) return rc;
    if ((rc = attention_setup()) != GEMM_OK) return rc;
    const KvPlan plan = kv_plan(v, b, q_heads, window, sms);
    void* scratch = nullptr;
    if (plan.scratch_bytes > 0 && !(scratch = scratch_alloc(plan.scratch_bytes, stream))) return GEMM_ERR_NO_MEMORY;
    int launches = 0;
    if (launch_kv_attention(v, KvRows{const_cast<void*>(Q), q_row_stride, q_head_stride},
                            KvRows{O, o_row_stride, o_head_stride}, static_cast<ElemType>(type), q_heads,
                            scale, causal != 0, window, b, plan, scratch, err, &launches, stream) != cudaSuccess)
        rc = GEMM_ERR_CUDA;
    for (int i = 0; i < launches; ++i) count_launch();
    if (scratch && cudaFreeAsync(scratch, stream) != cudaSuccess && rc == GEMM_OK) rc = GEMM_ERR_CUDA;
    return rc;
}

}  // extern "C"
