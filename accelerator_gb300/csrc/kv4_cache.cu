// kv4_cache.cu -- writing keys and values into the paged 4-bit cache and
// reading them back (layouts and rules in gemm.h).
//
// A token's keys (or values) of one head have a scale of their own, so that a
// token is written without those around it.  The unit of both directions is the
// part of one block of 16 tokens, head and operand that a call touches: one
// warp, whose lane (g, t) = (lane / 4, lane % 4) holds what it is about to
// write in whole pieces of a code block -- of the keys of tokens g and g + 8 the
// 8 dimensions from 8t on of each 32, of the values of tokens 2t, 2t + 1, 2t + 8
// and 2t + 9 those from 8g on of each 64 -- so that rows come in 16-byte loads,
// all in flight at once, and the largest magnitude of a row is found over 4 or 8
// lanes.
//
// 11000 tokens of 4 prompts, 8 heads of 128, bfloat16 (45 MB one way, 12 the other):
// 18 us to write and 13 us to read back out of a cold L2, 3.2 and 4.3 TB/s, where
// the measured copy rate would give 8.4 us each way.  Neither instructions nor memory
// are at their limit: SMs are at work for 77 and 70 % of the time (1.8 and 1.5 rounds
// of blocks), and then issue 0.61 instructions a cycle and scheduler (10.2 and 7.0 million
// in all) at half of their warps' places; of a warp's waits 28 and 31 % are for its
// loads, which come behind the search for its part, then for the ALU pipe.  The
// raising of tiny rows inside the pairs' arithmetic, without a branch around a row's,
// cost 1.3 us; a block that goes through all heads of its part saves searches and has
// fewer warps: 21.9 and 14.7 us.
#include "kernels.h"
#include "kv_part.cuh"
#include "lowbit.cuh"

namespace libgemm {
namespace {

constexpr float kTiny = 1.1754943508222875e-38f;   // 2^-126
constexpr int kWarps = 8, kThreads = kWarps * 32;  // of a CTA: all of one block of tokens
constexpr int kBlockLog2 = 4;

// A row's scale s = bf16(max|x| * (1 / 7)) and what its codes are made with.
struct Scale {
    float s, inv;      // s = 0: the codes are those of zeros
    uint16_t bits;
    bool up;           // s and the elements are taken times 2^64, inv times 2^-64
};
template <typename T>
__device__ __forceinline__ Scale scale_of(uint32_t top) {   // the bits of the largest magnitude
    Scale r;
    const __nv_bfloat16 sb = __float2bfloat16_rn(__fmul_rn(__uint_as_float(top), 1.0f / 7.0f));
    r.s = __bfloat162float(sb);
    r.bits = __bfloat16_as_ushort(sb);
    if (top >= 0x7F800000u) r.s = 0.0f, r.bits = 0x7FC0;   // NaN; the codes are those of zeros
    else if (r.s < kTiny) r.s = 0.0f, r.bits = 0;
    r.inv = r.s == 0.0f ? 0.0f : __frcp_rn(r.s);
    // (binary16's least s is above that)
    r.up = !std::is_same<T, __half>::value && r.s < 7.9e-31f && r.s > 0.0f;
    if (r.up) r.s *= 18446744073709551616.0f, r.inv *= 5.421010862427522e-20f;   // 2^64, 2^-64
    return r;
}

// Codes of eight neighbours, the nibble e of element e: x / s rounded to the
// nearest integer, ties to even.  The quotient has to be the correctly rounded
// one, for it is often halfway between two integers: from q = x * (1 / s) the
// residual x - q * s (exact in one fused multiply-add) gives it (Markstein 1990)
// as long as nothing underflows, hence `up` and `raise` (which is exact: a change
// of exponent, of values under 2^-96).  |x / s| stays under 7.04.
template <typename T>
__device__ __forceinline__ void raise(Eight<T>& x, const Scale& r) {
    if constexpr (!std::is_same<T, __half>::value) {
        if (r.up)
#pragma unroll
            for (int e = 0; e < 8; ++e) x.put(e, x.at(e) * 18446744073709551616.0f);
    }
}

template <typename T>
__device__ __forceinline__ uint32_t nibbles_of(const Eight<T>& x, const Scale& r) {
    const float2 inv = make_float2(r.inv, r.inv), minus = make_float2(-r.s, -r.s);
    const float2 to_nibble = make_float2(12582920.0f, 12582920.0f);   // 1.5 * 2^23 + 8: rounds, and leaves u in the low byte
    float2 u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = make_float2(x.at(2 * i), x.at(2 * i + 1));
        const float2 q = __fmul2_rn(v, inv);
        u[i] = __fadd2_rn(__ffma2_rn(__ffma2_rn(q, minus, v), inv, q), to_nibble);
    }
    const uint32_t even = low_bytes(__float_as_uint(u[0].x), __float_as_uint(u[1].x), __float_as_uint(u[2].x), __float_as_uint(u[3].x));
    const uint32_t odd = low_bytes(__float_as_uint(u[0].y), __float_as_uint(u[1].y), __float_as_uint(u[2].y), __float_as_uint(u[3].y));
    return r.s == 0.0f ? 0x88888888u : even | odd << 4;
}

// The eight values c * s of a word of codes.
template <typename T>
__device__ __forceinline__ void store_values(T* to, uint32_t w, float s) {
    float2 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {   // u in the low fraction bits of 2^23
        auto one = [&](int e) { return __uint_as_float(((w >> (4 * e)) & 15u) | 0x4B000000u); };
        v[i] = __fmul2_rn(__fadd2_rn(make_float2(one(2 * i), one(2 * i + 1)), make_float2(-8388616.0f, -8388616.0f)), make_float2(s, s));
    }
    if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4*>(to)[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
        reinterpret_cast<float4*>(to)[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
    } else {
        *reinterpret_cast<uint4*>(to) = make_uint4(pack2<T>(v[0].x, v[0].y), pack2<T>(v[1].x, v[1].y),
                                                   pack2<T>(v[2].x, v[2].y), pack2<T>(v[3].x, v[3].y));
    }
}

// Where a unit's codes and scales lie in its page's record.
struct Place {
    uint8_t* codes;      // of the block's keys or values
    uint16_t* scales;    // of the block's tokens
    int64_t extent;      // of all records, for the checks
};
__device__ __forceinline__ Place place_of(const KvView& c, const Part& part, int h, bool values) {
    uint8_t* record = c.data + (part.page * c.heads + h) * c.record();
    const int half = c.dim / 2 << c.page_log2, page = 1 << c.page_log2;
    return Place{record + (values ? half : 0) + part.at * (c.dim / 2),
                 reinterpret_cast<uint16_t*>(record + 2 * half) + (values ? page : 0) + part.at, c.pages * c.heads * c.record()};
}

template <int BYTES>
__device__ __forceinline__ void store_chunk(uint8_t* to, const uint32_t* w) {
    if constexpr (BYTES == 16) *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
}
template <int BYTES>
__device__ __forceinline__ void load_chunk(const uint8_t* from, uint32_t* w) {
    if constexpr (BYTES == 16) {
        const uint4 v = *reinterpret_cast<const uint4*>(from);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(from);
        w[0] = v.x, w[1] = v.y;
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(KvView c, KvRows K, KvRows V, bool vec, KvBatch b, unsigned* err) {
    constexpr int kChunk = D / 8, kWords = D / 32;   // of a lane: bytes, words
    Part part;
    if (!find_part(c, b, kBlockLog2, blockIdx.x, err, part)) return;
    const int which = blockIdx.y * kWarps + threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int h = which >> 1;
    const bool values = which & 1;
    if (h >= c.heads) return;
    const KvRows& src = values ? V : K;
    const T* x = static_cast<const T*>(src.p) + part.row * src.row + h * src.head;
    [[maybe_unused]] const int64_t x_bytes = ((b.rows - 1) * src.row + (c.heads - 1) * src.head + D) * (int64_t)sizeof(T);
    const Place at = place_of(c, part, h, values);
    auto here = [&](int tok) { return tok >= part.begin && tok < part.end; };
    auto load = [&](int tok, int d) {
        Eight<T> e = {};
        const T* p = x + (int64_t)(tok - part.begin) * src.row + d;
        if (here(tok) && GEMM_DBG_OK(p, src.p, x_bytes, 8 * sizeof(T))) e = load_eight(p, vec);
        return e;
    };
    auto put_scale = [&](int tok, uint16_t bits) {
        if (here(tok) && GEMM_DBG_OK(at.scales + tok, c.data, at.extent, 2)) at.scales[tok] = bits;
    };
    if (!values) {
        Eight<T> held[2][kWords];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int i = 0; i < kWords; ++i) held[r][i] = load(8 * r + g, 32 * i + 8 * t);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            Tops<T> tops;
#pragma unroll
            for (int i = 0; i < kWords; ++i) tops.take(held[r][i]);
            uint32_t top = tops.all();
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            const Scale s = scale_of<T>(top);
            const int tok = 8 * r + g;
            uint32_t w[kWords];
#pragma unroll
            for (int i = 0; i < kWords; ++i) raise(held[r][i], s), w[i] = nibbles_of(held[r][i], s);
            uint8_t* to = at.codes + tok * (D / 2) + t * kChunk;
            if (here(tok) && GEMM_DBG_OK(to, c.data, at.extent, kChunk)) store_chunk<kChunk>(to, w);
            if (t == 0) put_scale(tok, s.bits);
        }
    } else {
        Eight<T> held[2][2][D / 64];   // tokens 8r + 2t + o
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int o = 0; o < 2; ++o)
#pragma unroll
                for (int i = 0; i < D / 64; ++i) held[r][o][i] = load(8 * r + 2 * t + o, 64 * i + 8 * g);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            uint32_t own[2][D / 64];   // each token's words
#pragma unroll
            for (int o = 0; o < 2; ++o) {
                Tops<T> tops;
#pragma unroll
                for (int i = 0; i < D / 64; ++i) tops.take(held[r][o][i]);
                uint32_t top = tops.all();
#pragma unroll
                for (int m = 4; m < 32; m *= 2) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));
                const Scale s = scale_of<T>(top);
#pragma unroll
                for (int i = 0; i < D / 64; ++i) raise(held[r][o][i], s), own[o][i] = nibbles_of(held[r][o][i], s);
                if (g == 0) put_scale(8 * r + 2 * t + o, s.bits);
            }
            // four dimensions of both tokens to a word
            uint32_t w[kWords];
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                w[2 * i] = __byte_perm(own[0][i], own[1][i], 0x5410);
                w[2 * i + 1] = __byte_perm(own[0][i], own[1][i], 0x7632);
            }
            const int tok = 8 * r + 2 * t;
            uint8_t* to = at.codes + r * (4 * D) + lane * kChunk;
            if (!GEMM_DBG_OK(to, c.data, at.extent, kChunk)) continue;
            if (here(tok) && here(tok + 1)) store_chunk<kChunk>(to, w);
            else if (here(tok) || here(tok + 1)) {   // a token's halves of the words alone
                const int o = here(tok) ? 0 : 1;
#pragma unroll
                for (int i = 0; i < kWords; ++i) reinterpret_cast<uint16_t*>(to)[2 * i + o] = (uint16_t)(w[i] >> (16 * o));
            }
        }
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(KvView c, T* __restrict__ K, T* __restrict__ V, KvBatch b, unsigned* err) {
    constexpr int kChunk = D / 8, kWords = D / 32;
    Part part;
    if (!find_part(c, b, kBlockLog2, blockIdx.x, err, part)) return;
    const int which = blockIdx.y * kWarps + threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int h = which >> 1;
    const bool values = which & 1;
    if (h >= c.heads) return;
    T* out = values ? V : K;
    const int64_t step = (int64_t)c.heads * D;
    T* to = out + part.row * step + h * D;
    [[maybe_unused]] const int64_t out_bytes = b.rows * step * (int64_t)sizeof(T);
    const Place at = place_of(c, part, h, values);
    uint32_t w[2][kWords] = {};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const uint8_t* from = at.codes + (values ? r * (4 * D) + lane * kChunk : (8 * r + g) * (D / 2) + t * kChunk);
        if (GEMM_DBG_OK(from, c.data, at.extent, kChunk)) load_chunk<kChunk>(from, w[r]);
    }
    auto put = [&](int tok, int d, uint32_t word) {
        if (tok < part.begin || tok >= part.end || !GEMM_DBG_OK(at.scales + tok, c.data, at.extent, 2)) return;
        T* p = to + (tok - part.begin) * step + d;
        if (GEMM_DBG_OK(p, out, out_bytes, 8 * sizeof(T))) store_values(p, word, __uint_as_float((uint32_t)at.scales[tok] << 16));
    };
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if (!values) put(8 * r + g, 32 * i + 8 * t, w[r][i]);
            else put(8 * r + 2 * t + (i & 1), 64 * (i / 2) + 8 * g, __byte_perm(w[r][i & ~1], w[r][i | 1], i & 1 ? 0x7632 : 0x5410));
        }
}

dim3 grid_of(const KvView& c, const KvBatch& b) {
    return dim3((unsigned)((b.rows >> kBlockLog2) + 2 * (int64_t)b.sequences), (unsigned)((2 * c.heads + kWarps - 1) / kWarps));
}

template <typename T>
void append(const KvView& c, const KvRows& K, const KvRows& V, const KvBatch& b, unsigned* err, cudaStream_t stream) {
    auto by16 = [](const KvRows& r) {
        const int64_t es = sizeof(T);
        return (reinterpret_cast<uintptr_t>(r.p) & 15u) == 0 && r.row * es % 16 == 0 && r.head * es % 16 == 0;
    };
    const bool vec = by16(K) && by16(V);
    if (c.dim == 64) kv4_append_kernel<T, 64><<<grid_of(c, b), kThreads, 0, stream>>>(c, K, V, vec, b, err);
    else kv4_append_kernel<T, 128><<<grid_of(c, b), kThreads, 0, stream>>>(c, K, V, vec, b, err);
}

template <typename T>
void read(const KvView& c, void* K, void* V, const KvBatch& b, unsigned* err, cudaStream_t stream) {
    T *k = static_cast<T*>(K), *v = static_cast<T*>(V);
    if (c.dim == 64) kv4_read_kernel<T, 64><<<grid_of(c, b), kThreads, 0, stream>>>(c, k, v, b, err);
    else kv4_read_kernel<T, 128><<<grid_of(c, b), kThreads, 0, stream>>>(c, k, v, b, err);
}

}  // namespace

LIBGEMM_DEBUG_READER(kv4_cache_debug_flags)

cudaError_t launch_kv4_append(const KvView& c, const KvRows& K, const KvRows& V, ElemType type,
                              const KvBatch& b, unsigned* err, cudaStream_t stream) {
    if (type == ElemType::kF32) append<float>(c, K, V, b, err, stream);
    else if (type == ElemType::kBF16) append<__nv_bfloat16>(c, K, V, b, err, stream);
    else append<__half>(c, K, V, b, err, stream);
    return cudaGetLastError();
}

cudaError_t launch_kv4_read(const KvView& c, void* K, void* V, ElemType type, const KvBatch& b,
                            unsigned* err, cudaStream_t stream) {
    if (type == ElemType::kF32) read<float>(c, K, V, b, err, stream);
    else if (type == ElemType::kBF16) read<__nv_bfloat16>(c, K, V, b, err, stream);
    else read<__half>(c, K, V, b, err, stream);
    return cudaGetLastError();
}

}  // namespace libgemm
