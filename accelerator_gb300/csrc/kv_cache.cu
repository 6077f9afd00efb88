// kv_cache.cu -- writing keys and values into the paged 8-bit cache and
// reading them back (layouts and rules in gemm.h).
//
// A page's codes of one head share one scale, so what is written together is
// a page: one CTA takes the new tokens of one (sequence, page, head) of the
// keys or the values.  Sequences and pages are found from the row offsets on
// the device; a launch has one unit for each page that could be touched.
#include "kernels.h"
#include "lowbit.cuh"

namespace libgemm {
namespace {

constexpr float kTiny = 1.1754943508222875e-38f;   // 2^-126
constexpr int kThreads = 128;

__device__ __forceinline__ uint8_t code_of(float x, float inv) {
    const float c = fminf(fmaxf(rintf(__fmul_rn(x, inv)), -127.0f), 127.0f);
    return (uint8_t)((int)c + 128);
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    kv_append_kernel(KvView c, KvRows K, KvRows V, KvBatch b, unsigned* err) {
    __shared__ uint32_t s_top;
    const int P = 1 << c.page_log2, tid = threadIdx.x;
    const int h = blockIdx.y >> 1;
    const bool values = blockIdx.y & 1;
    const KvRows& src = values ? V : K;
    uint8_t* codes = values ? c.v : c.k;
    float* scales = values ? c.vs : c.ks;
    const Starts starts{b.starts, b.sequences, b.rows};
    const int64_t u = blockIdx.x;
    // Sequence q's pages are units floor(starts[q] / P) + 2q + j: T rows touch
    // at most floor(T / P) + 2 pages, which is how far apart these are.
    const int q = last_not_above(b.sequences, u, [&](int i) { return (starts.at(i) >> c.page_log2) + 2 * (int64_t)i; });
    const int64_t row0 = starts.at(q), count = starts.at(q + 1) - row0;
    const bool report = tid == 0 && blockIdx.y == 0;
    if (!starts.good(q)) {
        if (report) atomicOr(err, kErrIndex);
        return;
    }
    const int64_t first = __ldg(b.at + q), j = u - (row0 >> c.page_log2) - 2 * (int64_t)q;
    if (count == 0) return;
    if (first < 0 || first + count > (b.width << c.page_log2)) {
        if (report) atomicOr(err, kErrIndex);
        return;
    }
    const int64_t blk = (first >> c.page_log2) + j, lo = blk << c.page_log2;
    if (lo >= first + count) return;
    const int64_t page = __ldg(b.table + q * b.width + blk);
    if (page < 0 || page >= c.pages) {
        if (report) atomicOr(err, kErrIndex);
        return;
    }
    const int begin = (int)(first > lo ? first - lo : 0);                    // first new token of the page
    const int end = (int)(first + count - lo < P ? first + count - lo : P);
    const T* x = static_cast<const T*>(src.p) + (row0 + lo + begin - first) * src.row + h * src.head;
    [[maybe_unused]] const int64_t x_bytes =
        ((b.rows - 1) * src.row + (c.heads - 1) * src.head + c.dim) * (int64_t)sizeof(T);
    [[maybe_unused]] const int64_t code_bytes = c.pages * c.heads * ((int64_t)c.dim << c.page_log2);
    const int dim = c.dim, n = (end - begin) * dim;
    uint32_t m = 0;
    for (int i = tid; i < n; i += kThreads) {
        const T* p = x + i / dim * src.row + i % dim;
        if (GEMM_DBG_OK(p, src.p, x_bytes, sizeof(T))) m = max(m, __float_as_uint(to_float(*p)) & 0x7FFFFFFFu);
    }
    if (tid == 0) s_top = 0;
    __syncthreads();
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if (tid % 32 == 0) atomicMax(&s_top, m);
    __syncthreads();
    m = s_top;
    float* sp = scales + page * c.heads + h;
    if (!GEMM_DBG_OK(sp, scales, c.pages * c.heads * 4, 4)) return;
    const float before = begin > 0 ? *sp : 0.0f;
    float s = fmaxf(before, __fdiv_rn(__uint_as_float(m), 127.0f));
    const bool bad = m >= 0x7F800000u || before != before;
    const float inv = bad || s < kTiny ? 0.0f : __fdiv_rn(1.0f, s);
    __syncthreads();   // every thread has read the old scale
    if (tid == 0) *sp = bad ? __uint_as_float(0x7FC00000u) : s;
    uint8_t* out = codes + ((page * c.heads + h) << c.page_log2) * dim;
    for (int i = tid; i < n; i += kThreads) {
        const T* p = x + i / dim * src.row + i % dim;
        uint8_t* o = out + begin * dim + i;
        if (GEMM_DBG_OK(p, src.p, x_bytes, sizeof(T)) && GEMM_DBG_OK(o, codes, code_bytes, 1))
            *o = bad ? 128 : code_of(to_float(*p), inv);
    }
    if (!bad && before < s) {
        const float r = __fmul_rn(before, inv);
        for (int i = tid; i < begin * dim; i += kThreads)
            if (GEMM_DBG_OK(out + i, codes, code_bytes, 1)) out[i] = (uint8_t)((int)rintf(__fmul_rn((float)((int)out[i] - 128), r)) + 128);
    }
}

// Each thread turns 16 codes of one row and head into values.
template <typename T>
__global__ void __launch_bounds__(256)
    kv_read_kernel(KvView c, T* __restrict__ K, T* __restrict__ V, KvBatch b, unsigned* err) {
    const int chunks = c.dim / 16;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t per_row = (int64_t)c.heads * chunks;
    if (i >= b.rows * per_row) return;
    const int64_t row = i / per_row;
    const int rest = (int)(i - row * per_row), h = rest / chunks, d = rest % chunks * 16;
    const Starts starts{b.starts, b.sequences, b.rows};
    const int q = last_not_above(b.sequences, row, [&](int j) { return starts.at(j); });
    const int64_t pos = (int64_t)__ldg(b.at + q) + row - starts.at(q), blk = pos >> c.page_log2;
    bool ok = starts.good(q) && row >= starts.at(q) && row < starts.at(q + 1) && pos >= 0 && blk < b.width;
    const int64_t page = ok ? __ldg(b.table + q * b.width + blk) : -1;
    ok = ok && page >= 0 && page < c.pages;
    if (!ok) {
        atomicOr(err, kErrIndex);
        return;
    }
    const int64_t ph = page * c.heads + h;
    const int64_t from = ((ph << c.page_log2) + (pos & ((1 << c.page_log2) - 1))) * c.dim + d;
    const int64_t to = (row * c.heads + h) * c.dim + d;
    [[maybe_unused]] const int64_t code_bytes = c.pages * c.heads * ((int64_t)c.dim << c.page_log2);
    [[maybe_unused]] const int64_t out_bytes = b.rows * c.heads * c.dim * (int64_t)sizeof(T);
#pragma unroll
    for (int o = 0; o < 2; ++o) {
        const uint8_t* codes = o ? c.v : c.k;
        T* out = (o ? V : K) + to;
        const float s = __ldg((o ? c.vs : c.ks) + ph);
        if (!GEMM_DBG_OK(codes + from, codes, code_bytes, 16) || !GEMM_DBG_OK(out, o ? V : K, out_bytes, 16 * sizeof(T))) continue;
        const uint4 w = *reinterpret_cast<const uint4*>(codes + from);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = __fmul_rn((float)((int)((ws[e / 4] >> (8 * (e % 4))) & 255u) - 128), s);
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                reinterpret_cast<float4*>(out)[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        } else {
#pragma unroll
            for (int e = 0; e < 2; ++e)
                reinterpret_cast<uint4*>(out)[e] =
                    make_uint4(pack2<T>(v[8 * e], v[8 * e + 1]), pack2<T>(v[8 * e + 2], v[8 * e + 3]),
                               pack2<T>(v[8 * e + 4], v[8 * e + 5]), pack2<T>(v[8 * e + 6], v[8 * e + 7]));
        }
    }
}

}  // namespace

LIBGEMM_DEBUG_READER(kv_cache_debug_flags)

cudaError_t launch_kv_append(const KvView& c, const KvRows& K, const KvRows& V, ElemType type,
                             const KvBatch& b, unsigned* err, cudaStream_t stream) {
    const dim3 grid((unsigned)((b.rows >> c.page_log2) + 2 * (int64_t)b.sequences), (unsigned)(2 * c.heads));
    if (type == ElemType::kF32) kv_append_kernel<float><<<grid, kThreads, 0, stream>>>(c, K, V, b, err);
    else if (type == ElemType::kBF16) kv_append_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(c, K, V, b, err);
    else kv_append_kernel<__half><<<grid, kThreads, 0, stream>>>(c, K, V, b, err);
    return cudaGetLastError();
}

cudaError_t launch_kv_read(const KvView& c, void* K, void* V, ElemType type, const KvBatch& b,
                           unsigned* err, cudaStream_t stream) {
    const unsigned grid = (unsigned)((b.rows * c.heads * (c.dim / 16) + 255) / 256);
    if (type == ElemType::kF32)
        kv_read_kernel<float><<<grid, 256, 0, stream>>>(c, static_cast<float*>(K), static_cast<float*>(V), b, err);
    else if (type == ElemType::kBF16)
        kv_read_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(c, static_cast<__nv_bfloat16*>(K), static_cast<__nv_bfloat16*>(V), b, err);
    else
        kv_read_kernel<__half><<<grid, 256, 0, stream>>>(c, static_cast<__half*>(K), static_cast<__half*>(V), b, err);
    return cudaGetLastError();
}

}  // namespace libgemm
