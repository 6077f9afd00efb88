// kv_cache.cu -- writing keys and values into the paged 8-bit cache and
// reading them back (layouts and rules in gemm.h).
//
// A page's codes of one head share one scale, so the unit of both directions
// is the part of one (sequence, page, head) of the keys or the values that a
// call touches: one CTA.  Sequences and pages are found from the row offsets
// on the device; a launch has one unit for each page that could be touched.
// Every thread has all of its loads in flight, 8 elements each, before it uses
// the first, and the new elements stay in registers between the search for
// their largest and the rounding.  11000 ragged tokens of 8 heads of 128: 18 us
// to write (3.7 TB/s; at 2.9 instructions a cycle, so bound by them as much as
// by memory) and 13 us to read back; one token for each of 64 sequences 8 and 10
// us, which are the chains of loads from offset to page to scale to code.
#include "kernels.h"
#include "kv_part.cuh"
#include "lowbit.cuh"

namespace libgemm {
namespace {

constexpr float kTiny = 1.1754943508222875e-38f;   // 2^-126
constexpr int kThreads = 256;

// Codes of four values: rint(x * f) + 128 as bytes.  |x * f| stays under 127.5:
// f is 1 / s and s at least max|x| * (1 / 127), but for three roundings.
__device__ __forceinline__ uint32_t codes_of(float2 a, float2 b, float f) {
    // single products: a packed one and the sum after it become one operation, without the rounding between them
    const float2 to_byte = make_float2(12583040.0f, 12583040.0f);   // 1.5 * 2^23 + 128
    return low_bytes(__fadd2_rn(make_float2(__fmul_rn(a.x, f), __fmul_rn(a.y, f)), to_byte),
                     __fadd2_rn(make_float2(__fmul_rn(b.x, f), __fmul_rn(b.y, f)), to_byte));
}
// Bytes i and i + 1 of a word of codes as c, exactly: u in the low fraction bits of 2^23.
__device__ __forceinline__ float2 values_of(uint32_t w, int i) {
    return __fadd2_rn(make_float2(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440 | i)),
                                  __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440 | (i + 1)))),
                      make_float2(-8388736.0f, -8388736.0f));
}

// UNITS groups of 8 elements a thread: a page's elements / 8 / kThreads.
template <typename T, int UNITS>
__global__ void __launch_bounds__(kThreads)
    kv_append_kernel(KvView c, KvRows K, KvRows V, bool vec, KvBatch b, unsigned* err) {
    __shared__ uint32_t s_top[kThreads / 32];
    const int tid = threadIdx.x, h = blockIdx.y >> 1;
    const bool values = blockIdx.y & 1;
    const KvRows& src = values ? V : K;
    uint8_t* codes = values ? c.v : c.k;
    float* scales = values ? c.vs : c.ks;
    Part part;
    if (!find_part(c, b, c.page_log2, blockIdx.x, err, part)) return;
    const int row_log2 = c.dim == 64 ? 3 : 4, n = (part.end - part.begin) << row_log2;   // groups of a row; in all
    const T* x = static_cast<const T*>(src.p) + part.row * src.row + h * src.head;
    [[maybe_unused]] const int64_t x_bytes =
        ((b.rows - 1) * src.row + (c.heads - 1) * src.head + c.dim) * (int64_t)sizeof(T);
    [[maybe_unused]] const int64_t code_bytes = c.pages * c.heads * ((int64_t)c.dim << c.page_log2);
    float* sp = scales + part.page * c.heads + h;
    if (!GEMM_DBG_OK(sp, scales, c.pages * c.heads * 4, 4)) return;
    const float before = part.begin > 0 ? *sp : 0.0f;

    Eight<T> held[UNITS] = {};
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
        const int e = tid + i * kThreads;
        if (i * kThreads >= n) break;
        const T* p = x + (int64_t)(e >> row_log2) * src.row + (e & ((1 << row_log2) - 1)) * 8;
        if (e < n && GEMM_DBG_OK(p, src.p, x_bytes, 8 * sizeof(T))) held[i] = load_eight(p, vec);
    }
    Tops<T> tops;
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
        if (i * kThreads >= n) break;
        tops.take(held[i]);
    }
    uint32_t m = __reduce_max_sync(0xFFFFFFFFu, tops.all());
    if (tid % 32 == 0) s_top[tid / 32] = m;
    __syncthreads();   // also: every thread has read the old scale
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) m = max(m, s_top[i]);
    const float s = fmaxf(before, __fmul_rn(__uint_as_float(m), 1.0f / 127.0f));
    const bool bad = m >= 0x7F800000u || before != before;
    const float inv = bad || s < kTiny ? 0.0f : __fdiv_rn(1.0f, s);
    if (tid == 0) *sp = bad ? __uint_as_float(0x7FC00000u) : s;
    uint8_t* out = codes + ((part.page * c.heads + h) << c.page_log2) * c.dim;
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
        const int e = tid + i * kThreads;
        uint8_t* o = out + part.begin * c.dim + e * 8;
        if (e >= n || !GEMM_DBG_OK(o, codes, code_bytes, 8)) break;
        const Eight<T>& x = held[i];
        uint2 w = make_uint2(codes_of(make_float2(x.at(0), x.at(1)), make_float2(x.at(2), x.at(3)), inv),
                             codes_of(make_float2(x.at(4), x.at(5)), make_float2(x.at(6), x.at(7)), inv));
        if (bad) w = make_uint2(0x80808080u, 0x80808080u);
        *reinterpret_cast<uint2*>(o) = w;
    }
    if (!bad && before < s) {   // the scale grew: the page's older codes follow
        const float r = __fmul_rn(before, inv);
        for (int e = tid; e < part.begin << row_log2; e += kThreads) {
            uint2* o = reinterpret_cast<uint2*>(out) + e;
            if (!GEMM_DBG_OK(o, codes, code_bytes, 8)) continue;
            const uint2 w = *o;
            *o = make_uint2(codes_of(values_of(w.x, 0), values_of(w.x, 2), r), codes_of(values_of(w.y, 0), values_of(w.y, 2), r));
        }
    }
}

template <typename T, int UNITS>
__global__ void __launch_bounds__(kThreads)
    kv_read_kernel(KvView c, T* __restrict__ K, T* __restrict__ V, KvBatch b, unsigned* err) {
    const int tid = threadIdx.x, h = blockIdx.y >> 1;
    const bool values = blockIdx.y & 1;
    Part part;
    if (!find_part(c, b, c.page_log2, blockIdx.x, err, part)) return;
    const uint8_t* codes = values ? c.v : c.k;
    const float* scales = values ? c.vs : c.ks;
    T* out = values ? V : K;
    const int row_log2 = c.dim == 64 ? 3 : 4, n = (part.end - part.begin) << row_log2;   // groups of a row; in all
    const int64_t ph = part.page * c.heads + h;
    const uint8_t* from = codes + ((ph << c.page_log2) + part.begin) * c.dim;
    T* to = out + (part.row * c.heads + h) * c.dim;
    [[maybe_unused]] const int64_t code_bytes = c.pages * c.heads * ((int64_t)c.dim << c.page_log2);
    [[maybe_unused]] const int64_t out_bytes = b.rows * c.heads * c.dim * (int64_t)sizeof(T);
    if (!GEMM_DBG_OK(scales + ph, scales, c.pages * c.heads * 4, 4)) return;
    const float s = scales[ph];
    uint2 held[UNITS] = {};
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
        const int e = tid + i * kThreads;
        if (e < n && GEMM_DBG_OK(from + e * 8, codes, code_bytes, 8)) held[i] = *(reinterpret_cast<const uint2*>(from) + e);
    }
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
        const int e = tid + i * kThreads;
        T* o = to + (int64_t)(e >> row_log2) * c.heads * c.dim + (e & ((1 << row_log2) - 1)) * 8;
        if (e >= n || !GEMM_DBG_OK(o, out, out_bytes, 8 * sizeof(T))) break;
        float2 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __fmul2_rn(values_of(j < 2 ? held[i].x : held[i].y, 2 * j & 3), make_float2(s, s));
        if constexpr (sizeof(T) == 4) {
            reinterpret_cast<float4*>(o)[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
            reinterpret_cast<float4*>(o)[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
        } else {
            *reinterpret_cast<uint4*>(o) = make_uint4(pack2<T>(v[0].x, v[0].y), pack2<T>(v[1].x, v[1].y),
                                                      pack2<T>(v[2].x, v[2].y), pack2<T>(v[3].x, v[3].y));
        }
    }
}

dim3 grid_of(const KvView& c, const KvBatch& b) {
    return dim3((unsigned)((b.rows >> c.page_log2) + 2 * (int64_t)b.sequences), (unsigned)(2 * c.heads));
}

// Calls f with the number of groups of 8 elements that a thread holds.
template <typename F>
void with_units(const KvView& c, F f) {
    const int units = (c.dim << c.page_log2) / (8 * kThreads);
    if (units <= 1) f(std::integral_constant<int, 1>());
    else if (units == 2) f(std::integral_constant<int, 2>());
    else if (units == 4) f(std::integral_constant<int, 4>());
    else f(std::integral_constant<int, 8>());
}

template <typename T>
void append(const KvView& c, const KvRows& K, const KvRows& V, const KvBatch& b, unsigned* err, cudaStream_t stream) {
    auto by16 = [](const KvRows& r) {
        const int64_t es = sizeof(T);
        return (reinterpret_cast<uintptr_t>(r.p) & 15u) == 0 && r.row * es % 16 == 0 && r.head * es % 16 == 0;
    };
    const bool vec = by16(K) && by16(V);
    with_units(c, [&](auto units) {
        kv_append_kernel<T, decltype(units)::value><<<grid_of(c, b), kThreads, 0, stream>>>(c, K, V, vec, b, err);
    });
}

template <typename T>
void read(const KvView& c, void* K, void* V, const KvBatch& b, unsigned* err, cudaStream_t stream) {
    with_units(c, [&](auto units) {
        kv_read_kernel<T, decltype(units)::value>
            <<<grid_of(c, b), kThreads, 0, stream>>>(c, static_cast<T*>(K), static_cast<T*>(V), b, err);
    });
}

}  // namespace

LIBGEMM_DEBUG_READER(kv_cache_debug_flags)

cudaError_t launch_kv_append(const KvView& c, const KvRows& K, const KvRows& V, ElemType type,
                             const KvBatch& b, unsigned* err, cudaStream_t stream) {
    if (type == ElemType::kF32) append<float>(c, K, V, b, err, stream);
    else if (type == ElemType::kBF16) append<__nv_bfloat16>(c, K, V, b, err, stream);
    else append<__half>(c, K, V, b, err, stream);
    return cudaGetLastError();
}

cudaError_t launch_kv_read(const KvView& c, void* K, void* V, ElemType type, const KvBatch& b,
                           unsigned* err, cudaStream_t stream) {
    if (type == ElemType::kF32) read<float>(c, K, V, b, err, stream);
    else if (type == ElemType::kBF16) read<__nv_bfloat16>(c, K, V, b, err, stream);
    else read<__half>(c, K, V, b, err, stream);
    return cudaGetLastError();
}

}  // namespace libgemm
