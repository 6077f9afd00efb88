// w4.cu -- products with 4-bit weights: C = X*W for a few rows X, the
// quantiser that makes W and its inverse.
//
// W stands for q_kn * s_gn: 4-bit integers q with one bfloat16 scale for each
// column and group of rows (32, 64 or 128).  The codes are laid out for the
// warp-wide matrix instruction: of a block of 16 columns x 64 rows, each lane
// holds in 16 bytes the elements that it feeds to four m16n8k16 instructions,
// the columns of W as the 16 rows of A.  The order of k inside an instruction
// is free as long as X follows it, so a lane's k are eight neighbours of each
// half of 32 rows, and its part of a row of X is one 16-byte load per half.
#include "kernels.h"
#include "lowbit.cuh"

namespace libgemm {
namespace {

constexpr float kTiny = 1.1754943508222875e-38f;   // 2^-126

struct W4 {
    uint32_t* codes;
    uint16_t* scales;
    int64_t K, N;
    int group, kb, groups;   // blocks of 64 rows, groups of rows
    int group_log2;
    __host__ __device__ int64_t nb() const { return (N + 15) / 16; }
};

// The quantiser takes tiles of 128 rows x 32 columns, a whole number of groups
// and blocks, with 128 threads of 32 elements each.
constexpr int kQRows = 128, kQCols = 32, kQThreads = 128;

__device__ __forceinline__ void tile_at(const W4& w, int64_t& k0, int64_t& n0) {
    const unsigned across = (unsigned)((w.N + kQCols - 1) / kQCols);
    k0 = (int64_t)(blockIdx.x / across) * kQRows;
    n0 = (int64_t)(blockIdx.x % across) * kQCols;
}

// ---- quantise ----------------------------------------------------------------
// A thread holds four neighbouring rows of eight columns, all loaded before
// the first is used, and a warp 32 rows, over which shuffles find the largest
// magnitude of a column (over warps, for longer groups, shared memory does);
// a word of codes is four rows of two columns eight apart, so a thread and its
// neighbour make half of it each and swap; the words leave in 16-byte pieces
// by way of shared memory.  Bound by instructions (19 an element, 2.8 a cycle)
// and the loads between two barriers, which eight small CTAs an SM overlap: 8192
// x 8192 bfloat16 in 49 us, 3.4 TB/s read and written (59 us as four CTAs of 256
// threads, 67 us with one element at a time and conversions to int).
template <typename T>
__global__ void __launch_bounds__(kQThreads, 8)
    w4_quantize_kernel(const T* __restrict__ B, int64_t ldb, bool vec, W4 w) {
    __shared__ uint32_t top[4][kQCols];
    __shared__ __align__(16) float scale[4][kQCols], inverse[4][kQCols];
    __shared__ __align__(16) uint32_t words[2 * 296];   // [16 columns][64 rows][128 words], spread over the banks
    int64_t k0, n0;
    tile_at(w, k0, n0);
    const int tid = threadIdx.x, c8 = tid % 4, r = tid / 4;   // a warp has 32 rows
    [[maybe_unused]] const int64_t b_bytes = ((w.K - 1) * ldb + w.N) * (int64_t)sizeof(T);
    Eight<T> x[4] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t k = k0 + 4 * r + i, n = n0 + 8 * c8;
        const T* p = B + k * ldb + n;
        if (k >= w.K || n >= w.N) continue;
        if (n + 8 <= w.N) {
            if (GEMM_DBG_OK(p, B, b_bytes, 8 * sizeof(T))) x[i] = load_eight(p, vec);
        } else {
            T part[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) part[j] = n + j < w.N && GEMM_DBG_OK(p + j, B, b_bytes, sizeof(T)) ? p[j] : from_float<T>(0.0f);
            x[i] = load_eight(part, false);
        }
    }
    Tops<T> tops;
#pragma unroll
    for (int i = 0; i < 4; ++i) tops.take(x[i]);
    tops.across(4);
    tops.across(8);
    tops.across(16);
    if (tid % 32 < 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j) top[tid / 32][8 * c8 + j] = tops.bits(j);
    }
    __syncthreads();
    {
        const int c = tid % kQCols, part = tid / kQCols, per = w.group / 32, first = part & ~(per - 1);
        uint32_t m = 0;
        for (int i = 0; i < per; ++i) m = max(m, top[first + i][c]);
        const __nv_bfloat16 sb = __float2bfloat16_rn(__fmul_rn(__uint_as_float(m), 1.0f / 7.0f));
        float s = __bfloat162float(sb);
        uint16_t bits = __bfloat16_as_ushort(sb);
        if (m >= 0x7F800000u) s = 0.0f, bits = 0x7FC0;   // NaN; the codes are 0
        else if (s < kTiny) s = 0.0f, bits = 0;
        scale[part][c] = s;
        inverse[part][c] = s == 0.0f ? 0.0f : __fdiv_rn(1.0f, s);
        const int64_t g = (k0 + part * 32) >> w.group_log2, n = n0 + c;
        if (part == first && k0 + part * 32 < w.K && n < w.nb() * 16) {
            uint16_t* p = w.scales + ((n / 16 * w.groups + g) * 8 + n % 8) * 2 + n % 16 / 8;
            if (GEMM_DBG_OK(p, w.scales, w.nb() * w.groups * 32, 2)) *p = bits;
        }
    }
    __syncthreads();
    // b / s rounded to the nearest integer: the quotient has to be the
    // correctly rounded one, for b / s is often halfway between two integers.
    // From t = b * (1 / s) the residual b - t * s (exact in one fused
    // multiply-add) gives it (Markstein 1990) as long as nothing underflows,
    // which needs s above about 2^-100: below, b and s are taken times 2^64.
    // |b / s| stays under 7.04, as s is at most 2^-8 below max|b| / 7.
    uint32_t mine[8];
    const int hi = c8 & 1, part = r / 8;
    float s8[8], inv8[8];
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
        *reinterpret_cast<float4*>(s8 + j) = *reinterpret_cast<const float4*>(&scale[part][8 * c8 + j]);
        *reinterpret_cast<float4*>(inv8 + j) = *reinterpret_cast<const float4*>(&inverse[part][8 * c8 + j]);
    }
    if constexpr (!std::is_same<T, __half>::value) {   // binary16's least s is above that
        bool tiny = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) tiny |= s8[j] < 7.9e-31f && s8[j] > 0.0f;
        if (tiny) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool up = s8[j] < 7.9e-31f && s8[j] > 0.0f;
                if (up) s8[j] *= 18446744073709551616.0f, inv8[j] *= 5.421010862427522e-20f;   // 2^64, 2^-64
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (up) x[i].put(j, x[i].at(j) * 18446744073709551616.0f);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float s = s8[j], inv = inv8[j];
        const float2 i2 = make_float2(inv, inv), n2 = make_float2(-s, -s), to_nibble = make_float2(12582920.0f, 12582920.0f);   // 1.5 * 2^23 + 8
        float2 u[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const float2 b = make_float2(x[2 * p].at(j), x[2 * p + 1].at(j));
            const float2 t = __fmul2_rn(b, i2);
            u[p] = __fadd2_rn(__ffma2_rn(__ffma2_rn(t, n2, b), i2, t), to_nibble);
        }
        // rows 0, 2, 1, 3 in the nibbles 0, 2, 4, 6
        const uint32_t v = low_bytes(__float_as_uint(u[0].x), __float_as_uint(u[1].x), __float_as_uint(u[0].y), __float_as_uint(u[1].y));
        mine[j] = (s == 0.0f ? 0x08080808u : v) << (4 * hi);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {   // the even thread keeps columns 0-3 of 8, the odd one 4-7
        const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, hi ? mine[j] : mine[j + 4], 1);
        const uint32_t word = (hi ? mine[j + 4] : mine[j]) | got;
        const int g = j + 4 * hi, t = (r >> 1) & 3, at = 4 * (4 * g + t) + 2 * ((r >> 3) & 1) + (r & 1);
        words[c8 / 2 * 296 + r / 16 * 144 + at + 16 * (at >> 6)] = word;
    }
    __syncthreads();
    {
        const int nbl = tid / 64, kbl = tid / 32 % 2, at = tid % 32 * 4;
        const int64_t nb = n0 / 16 + nbl, kb = k0 / 64 + kbl;
        uint32_t* p = w.codes + (nb * w.kb + kb) * 128 + at;
        if (nb < w.nb() && kb < w.kb && GEMM_DBG_OK(p, w.codes, w.nb() * w.kb * 512, 16))
            *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(&words[nbl * 296 + kbl * 144 + at + 16 * (at >> 6)]);
    }
}

// ---- dequantise --------------------------------------------------------------
// A warp takes 64 rows of eight blocks side by side.  Their words come in
// 16-byte pieces and pass through shared memory, so that a thread gets word 4t +
// j of each of a block's eight g: four rows of all of its 16 columns, and what
// it stores is a row's 16 neighbours, a warp's 128.  Bound by shared memory (the
// words' reads meet four to a bank) and the stores: 8192 x 8192 to bfloat16 in
// 29 us, 5.8 TB/s; in 16-byte stores 40 us, by single elements 37 us.
constexpr int kDWarps = 4, kDCols = 128, kDPad = 136;   // kDPad: words of a block in shared memory

// 32 bytes at once (32-byte aligned).
__device__ __forceinline__ void store32(void* p, const uint32_t (&r)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

template <typename T>
__global__ void __launch_bounds__(kDWarps * 32)
    w4_dequantize_kernel(W4 w, T* __restrict__ B, int64_t ldb, bool vec) {
    __shared__ __align__(16) uint32_t s_words[kDWarps][kDCols / 16][kDPad];
    __shared__ __align__(16) T s_rows[kDWarps][4][kDCols + 16 / sizeof(T)];   // where rows are not aligned
    const unsigned across = (unsigned)((w.N + kDCols - 1) / kDCols);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t kb = (int64_t)(blockIdx.x / across) * kDWarps + warp, nb0 = (int64_t)(blockIdx.x % across) * (kDCols / 16);
    if (kb >= w.kb) return;
    uint4 piece[8] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint4* p = reinterpret_cast<const uint4*>(w.codes + ((nb0 + i) * w.kb + kb) * 128) + lane;
        if (nb0 + i < w.nb() && GEMM_DBG_OK(p, w.codes, w.nb() * w.kb * 512, 16)) piece[i] = __ldg(p);
    }
    const int64_t nb = nb0 + lane / 4, n = nb * 16, n0 = nb0 * 16;
    const int t = lane % 4;
    uint32_t scales[2][8] = {};   // of columns g and g + 8 together, for both halves of the rows
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t k = kb * 64 + 32 * h;
        const uint16_t* sp = w.scales + (nb * w.groups + (k >> w.group_log2)) * 16;
        if (nb >= w.nb() || k >= w.K || !GEMM_DBG_OK(sp, w.scales, w.nb() * w.groups * 32, 32)) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint2 s2 = __ldg(reinterpret_cast<const uint2*>(sp) + i);
            scales[h][2 * i] = s2.x, scales[h][2 * i + 1] = s2.y;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(&s_words[warp][i][4 * lane]) = piece[i];
    __syncwarp();
    [[maybe_unused]] const int64_t b_bytes = ((w.K - 1) * ldb + w.N) * (int64_t)sizeof(T);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int h = j / 2;
        uint32_t words[8];
#pragma unroll
        for (int g = 0; g < 8; ++g) words[g] = s_words[warp][lane / 4][16 * g + 4 * t + j];
        const int64_t k = kb * 64 + 32 * h + 8 * t + 4 * (j % 2);
        T* to = B + k * ldb + n;
#pragma unroll
        for (int e = 0; e < 4; ++e, to += ldb) {
            float2 v[8];   // columns 2i, 2i + 1
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
                const int shift = 4 * (4 * (e & 1) + 2 * (e >> 1) + hi);
                auto one = [&](int g) { return __uint_as_float(((words[g] >> shift) & 15u) | 0x4B000000u); };
                auto scale = [&](int g) { return __uint_as_float(hi ? scales[h][g] & 0xFFFF0000u : scales[h][g] << 16); };
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[4 * hi + i] = __fmul2_rn(__fadd2_rn(make_float2(one(2 * i), one(2 * i + 1)), make_float2(-8388616.0f, -8388616.0f)),
                                               make_float2(scale(2 * i), scale(2 * i + 1)));
            }
            // the whole width in aligned pieces, or by way of shared memory
            if (vec && n0 + kDCols <= w.N) {
                if (k + e >= w.K || !GEMM_DBG_OK(to, B, b_bytes, 16 * sizeof(T))) continue;
                uint32_t r[sizeof(T) == 4 ? 2 : 1][8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if constexpr (sizeof(T) == 4) {
                        r[i / 4][2 * i % 8] = __float_as_uint(v[i].x);
                        r[i / 4][2 * i % 8 + 1] = __float_as_uint(v[i].y);
                    } else {
                        r[0][i] = pack2<T>(v[i].x, v[i].y);
                    }
                }
#pragma unroll
                for (int i = 0; i < (int)sizeof(T) / 2; ++i) store32(reinterpret_cast<uint8_t*>(to) + 32 * i, r[i]);
            } else {
                T* row = s_rows[warp][t] + 16 * (lane / 4);
#pragma unroll
                for (int i = 0; i < 8; ++i) row[2 * i] = from_float<T>(v[i].x), row[2 * i + 1] = from_float<T>(v[i].y);
                __syncwarp();
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int64_t kr = k - 8 * t + 8 * r + e;   // the row of the lanes with t = r
                    T* out = B + kr * ldb + n0;
#pragma unroll
                    for (int c = lane; c < kDCols; c += 32)
                        if (kr < w.K && n0 + c < w.N && GEMM_DBG_OK(out + c, B, b_bytes, sizeof(T))) out[c] = s_rows[warp][r][c];
                }
                __syncwarp();
            }
        }
    }
}

// ---- the product -------------------------------------------------------------
constexpr int kPWarps = 8;
constexpr int kAhead = 4;       // blocks of 64 rows whose codes a warp has in flight
constexpr int resident(int mt) { return mt <= 2 ? 2 : 1; }   // CTAs of an SM

// Four nibble pairs of a word as pairs of T holding q, exactly.
template <typename T>
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t (&a)[4]);
template <>
__device__ __forceinline__ void unpack8<__half>(uint32_t w, uint32_t (&a)[4]) {
    // u in the low four fraction bits of 1024 is 1024 + u, in the next four
    // of 64 it is 64 + u; less 1032 and 72 both are q = u - 8
    auto sub = [](uint32_t x, uint32_t y) {
        const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
        return *reinterpret_cast<const uint32_t*>(&h);
    };
    a[0] = sub((w & 0x000F000Fu) | 0x64006400u, 0x64086408u);
    a[1] = sub((w & 0x00F000F0u) | 0x54005400u, 0x54805480u);
    w >>= 8;
    a[2] = sub((w & 0x000F000Fu) | 0x64006400u, 0x64086408u);
    a[3] = sub((w & 0x00F000F0u) | 0x54005400u, 0x54805480u);
}
template <>
__device__ __forceinline__ void unpack8<__nv_bfloat16>(uint32_t w, uint32_t (&a)[4]) {
    // u in the low fraction bits of 128 is 128 + u; less 136 it is q
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t x = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u, y = 0x43084308u;
        const __nv_bfloat162 h = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x),
                                         *reinterpret_cast<const __nv_bfloat162*>(&y));
        a[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
}

// Eight neighbours of one row of X as four pairs, where rows are aligned to 8, 4 or 2 bytes.
template <typename T>
__device__ __forceinline__ uint4 load_x8(const T* p, int align) {
    if (align == 8) {
        const uint2 a = __ldg(reinterpret_cast<const uint2*>(p)), b = __ldg(reinterpret_cast<const uint2*>(p) + 1);
        return make_uint4(a.x, a.y, b.x, b.y);
    }
    if (align == 4) {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(p);
        return make_uint4(__ldg(q), __ldg(q + 1), __ldg(q + 2), __ldg(q + 3));
    }
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
    auto two = [&](int e) { return (uint32_t)__ldg(q + e) | (uint32_t)__ldg(q + e + 1) << 16; };
    return make_uint4(two(0), two(2), two(4), two(6));
}
// Eight neighbours x[k .. k + 7] of one row of X as four pairs; 0 past K.
template <typename T>
__device__ __noinline__ uint4 load_x8_edge(const T* row, int k, int K) {
    uint32_t r[4] = {0, 0, 0, 0};
    const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
    for (int i = 0; i < 8; ++i)
        if (k + i < K) r[i / 2] |= (uint32_t)__ldg(p + k + i) << (16 * (i & 1));
    return make_uint4(r[0], r[1], r[2], r[3]);
}

__device__ __forceinline__ uint4 load_once(const uint4* p) {   // streamed past L1, which is for X
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// A cluster of CTAs computes 32 * WN columns of C for 8 * MT rows: each CTA a
// range of the blocks of 64 rows of W, in which each of its warps takes every
// WK-th block of 32 columns (two blocks of 16, so that a part of X that is
// loaded serves both).  The sums are added up over the warps, then over the
// cluster's CTAs through distributed shared memory, always in that order.
//
// Bound by instructions and their latency, not by the codes' bytes: 100 a block
// of 64 x 16 with 16 rows, of which 44 turn codes into bfloat16 (half of them at
// half rate), 1.9 a cycle at 16 warps an SM.  16 x 16384 x 16384: 54 us, 2.56
// TB/s; 1 x 8192 x 8192: 14.4 us, 2.4 TB/s.  Three CTAs an SM with fewer loads
// in flight were slower (57 us), and so was a ring of bulk copies (76 us).
template <typename T, typename U, int MT, int WN, bool HALF>
__global__ void __launch_bounds__(kPWarps * 32, resident(MT))
    w4_gemm_kernel(const T* __restrict__ X, int64_t ldx, W4 w, U* __restrict__ C, int64_t ldc,
                   int64_t M, int splits, int64_t tiles_n, int align) {
    constexpr int WK = kPWarps / WN, kCols = 32 * WN, kRows = 8 * MT;
    __shared__ float part[WK][kRows][kCols + 4];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int wn = warp % WN, wk = warp / WN;
    const int rank = blockIdx.x % splits;
    const int64_t tile = blockIdx.x / splits, m0 = tile / tiles_n * kRows;
    const int64_t nb0 = (tile % tiles_n) * (2 * WN) + 2 * wn;
    const int per = (w.kb + splits - 1) / splits;
    const int kb0 = rank * per, kb1 = min(w.kb, kb0 + per);
    [[maybe_unused]] const int64_t code_bytes = w.nb() * w.kb * 512, scale_bytes = w.nb() * w.groups * 32;

    const uint4* codes[2];
    const uint16_t* scales[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        // past the last column the last block again, whose sums are not stored
        const int64_t nb = min(nb0 + b, w.nb() - 1);
        codes[b] = reinterpret_cast<const uint4*>(w.codes + nb * w.kb * 128) + lane;
        scales[b] = w.scales + nb * w.groups * 16 + 2 * g;
    }
    const T* rows[MT];   // past the last row that row again, likewise
#pragma unroll
    for (int m = 0; m < MT; ++m) rows[m] = X + min(m0 + 8 * m + g, M - 1) * ldx + 8 * t;
    uint4 q[kAhead][2];
    uint32_t s2[kAhead][2][HALF ? 2 : 1];
    const int group_shift = w.group == 128 ? 1 : 0;   // blocks of a group
    auto fetch = [&](int slot, int kb) {
        kb = min(kb, kb1 - 1);   // past the end the last block again, unused
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            if (GEMM_DBG_OK(codes[b] + kb * 32, w.codes, code_bytes, 16)) q[slot][b] = load_once(codes[b] + kb * 32);
#pragma unroll
            for (int h = 0; h < (HALF ? 2 : 1); ++h) {
                // a last half block past K has X = 0: any scale of the column will do
                const uint16_t* sp = scales[b] + (HALF ? min(2 * kb + h, w.groups - 1) : kb >> group_shift) * 16;
                if (GEMM_DBG_OK(sp, w.scales, scale_bytes, 4)) s2[slot][b][h] = __ldg(reinterpret_cast<const uint32_t*>(sp));
            }
        }
    };
    const int K = (int)w.K;
    [[maybe_unused]] const int64_t x_bytes = ((M - 1) * ldx + w.K) * (int64_t)sizeof(T);
    constexpr int kX = MT <= 2 ? 2 : 1;   // parts of X: with few rows the next block's are in flight too
    uint4 x[kX][2][MT];
    auto fetch_x = [&](int slot, int kb) {
        kb = min(kb, kb1 - 1);
        if (align == 16 && kb * 64 + 64 <= K) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const T* p = rows[m] + kb * 64 + 32 * h;
                    if (GEMM_DBG_OK(p, X, x_bytes, 16)) x[slot][h][m] = __ldg(reinterpret_cast<const uint4*>(p));
                }
        } else if (kb * 64 + 64 <= K) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const T* p = rows[m] + kb * 64 + 32 * h;
                    if (GEMM_DBG_OK(p, X, x_bytes, 16)) x[slot][h][m] = load_x8(p, align);
                }
        } else {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    x[slot][h][m] = load_x8_edge(rows[m], kb * 64 + 32 * h, K - 8 * t);
        }
    };
    float total[2][MT][4] = {};
    if (kb0 + wk < kb1) {
#pragma unroll
        for (int p = 0; p < kAhead; ++p) fetch(p, kb0 + wk + p * WK);
        if (kX == 2) fetch_x(0, kb0 + wk);
    }
    for (int kb = kb0 + wk; kb < kb1; kb += kAhead * WK) {
#pragma unroll
        for (int p = 0; p < kAhead; ++p) {
            const int at = kb + p * WK;
            if (at >= kb1) break;
            fetch_x((p + 1) % kX, kX == 2 ? at + WK : at);
            const int xs = p % kX;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const uint32_t words[4] = {q[p][b].x, q[p][b].y, q[p][b].z, q[p][b].w};
                float acc[MT][4] = {};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t a0[4], a1[4];
                    unpack8<T>(words[2 * h], a0);
                    unpack8<T>(words[2 * h + 1], a1);
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        mma_16816<T>(acc[m], a0[0], a0[1], a0[2], a0[3], x[xs][h][m].x, x[xs][h][m].y);
                        mma_16816<T>(acc[m], a1[0], a1[1], a1[2], a1[3], x[xs][h][m].z, x[xs][h][m].w);
                    }
                    if (HALF || h == 1) {
                        const uint32_t s = s2[p][b][HALF ? h : 0];
                        const float lo = __uint_as_float(s << 16), hi = __uint_as_float(s & 0xFFFF0000u);
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            total[b][m][0] = fmaf(acc[m][0], lo, total[b][m][0]);
                            total[b][m][1] = fmaf(acc[m][1], lo, total[b][m][1]);
                            total[b][m][2] = fmaf(acc[m][2], hi, total[b][m][2]);
                            total[b][m][3] = fmaf(acc[m][3], hi, total[b][m][3]);
                            acc[m][0] = acc[m][1] = acc[m][2] = acc[m][3] = 0.0f;
                        }
                    }
                }
            }
            fetch(p, at + kAhead * WK);
        }
    }
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                part[wk][8 * m + 2 * t + (e & 1)][32 * wn + 16 * b + 8 * (e >> 1) + g] = total[b][m][e];
    __syncthreads();
    [[maybe_unused]] const int64_t c_bytes = ((M - 1) * ldc + w.N) * (int64_t)sizeof(U);
    auto store = [&](int i, float v) {
        const int64_t row = m0 + i / kCols, col = (nb0 - 2 * wn) * 16 + i % kCols;
        if (row >= M || col >= w.N) return;
        U* dst = C + row * ldc + col;
        if (GEMM_DBG_OK(dst, C, c_bytes, sizeof(U))) *dst = from_float<U>(v);
    };
    for (int i = threadIdx.x; i < kRows * kCols; i += kPWarps * 32) {
        float v = part[0][i / kCols][i % kCols];
#pragma unroll
        for (int p = 1; p < WK; ++p) v += part[p][i / kCols][i % kCols];
        if (splits == 1) store(i, v);
        else part[0][i / kCols][i % kCols] = v;
    }
    if (splits == 1) return;
    cluster_sync();
    const int share = (kRows * kCols + splits - 1) / splits;
    for (int i = rank * share + threadIdx.x; i < min(kRows * kCols, (rank + 1) * share); i += kPWarps * 32) {
        const uint32_t at = smem_u32(&part[0][i / kCols][i % kCols]);
        float v = ld_cluster_f32(mapa_shared(at, 0));
        for (int p = 1; p < splits; ++p) v += ld_cluster_f32(mapa_shared(at, p));
        store(i, v);
    }
    cluster_sync();   // no CTA leaves while another reads its sums
}

W4 view(const void* codes, const void* scales, int64_t K, int64_t N, int group) {
    return W4{const_cast<uint32_t*>(static_cast<const uint32_t*>(codes)),
              const_cast<uint16_t*>(static_cast<const uint16_t*>(scales)), K, N, group,
              (int)((K + 63) / 64), (int)((K + group - 1) / group), group == 32 ? 5 : group == 64 ? 6 : 7};
}

template <typename T, typename U, int MT, int WN, bool HALF>
cudaError_t launch_product(const T* X, int64_t ldx, const W4& w, U* C, int64_t ldc, int64_t M,
                           int align, int num_sms, cudaStream_t stream) {
    constexpr int WK = kPWarps / WN;
    const int64_t tiles_n = (w.nb() + 2 * WN - 1) / (2 * WN), tiles = tiles_n * ((M + 8 * MT - 1) / (8 * MT));
    // The blocks of rows are shared over a cluster of the size for which the
    // rounds of resident CTAs take least, a round costing the blocks of a warp
    // and about five more to start and to add up.
    const int64_t slots = (int64_t)num_sms * resident(MT);
    int splits = 1;
    int64_t least = INT64_MAX;
    for (int s = 1; s <= 8 && (s == 1 || s * WK <= w.kb); ++s) {
        const int64_t per = (w.kb + s - 1) / s;
        const int64_t cost = (tiles * s + slots - 1) / slots * ((per + WK - 1) / WK + 5);
        if (cost < least) least = cost, splits = s;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * splits));
    cfg.blockDim = dim3(kPWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)splits;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = splits > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, w4_gemm_kernel<T, U, MT, WN, HALF>, X, ldx, w, C, ldc, M, splits, tiles_n, align);
}

// More rows go with more columns to a CTA: X is read once for every tile of
// columns, 2 * rows bytes beside each column's half byte of codes.
template <typename T, typename U>
cudaError_t launch_by_rows(const T* X, int64_t ldx, const W4& w, U* C, int64_t ldc, int64_t M,
                           int align, int num_sms, cudaStream_t stream) {
    auto go = [&](auto mt, auto wn) {
        constexpr int MT = decltype(mt)::value, WN = decltype(wn)::value;
        return w.group == 32 ? launch_product<T, U, MT, WN, true>(X, ldx, w, C, ldc, M, align, num_sms, stream)
                             : launch_product<T, U, MT, WN, false>(X, ldx, w, C, ldc, M, align, num_sms, stream);
    };
    using std::integral_constant;
    if (M <= 2) return go(integral_constant<int, 1>(), integral_constant<int, 1>());
    if (M <= 8) return go(integral_constant<int, 1>(), integral_constant<int, 2>());
    if (M <= 16) return go(integral_constant<int, 2>(), integral_constant<int, 4>());
    return go(integral_constant<int, 4>(), integral_constant<int, 4>());
}

}  // namespace

LIBGEMM_DEBUG_READER(w4_debug_flags)

cudaError_t launch_w4_quantize(const void* B, int64_t ldb, ElemType type, int64_t K, int64_t N,
                               int group, void* codes, void* scales, cudaStream_t stream) {
    const W4 w = view(codes, scales, K, N, group);
    const unsigned grid = (unsigned)(((K + kQRows - 1) / kQRows) * ((N + kQCols - 1) / kQCols));
    const int64_t es = type == ElemType::kF32 ? 4 : 2;
    const bool vec = (reinterpret_cast<uintptr_t>(B) & 15u) == 0 && ldb * es % 16 == 0;
    if (type == ElemType::kF32)
        w4_quantize_kernel<float><<<grid, kQThreads, 0, stream>>>(static_cast<const float*>(B), ldb, vec, w);
    else if (type == ElemType::kBF16)
        w4_quantize_kernel<__nv_bfloat16><<<grid, kQThreads, 0, stream>>>(static_cast<const __nv_bfloat16*>(B), ldb, vec, w);
    else
        w4_quantize_kernel<__half><<<grid, kQThreads, 0, stream>>>(static_cast<const __half*>(B), ldb, vec, w);
    return cudaGetLastError();
}

cudaError_t launch_w4_dequantize(const void* codes, const void* scales, int64_t K, int64_t N,
                                 int group, void* B, int64_t ldb, ElemType type,
                                 cudaStream_t stream) {
    const W4 w = view(codes, scales, K, N, group);
    const unsigned grid = (unsigned)(((K + kDWarps * 64 - 1) / (kDWarps * 64)) * ((N + kDCols - 1) / kDCols));
    const int64_t es = type == ElemType::kF32 ? 4 : 2;
    const bool vec = (reinterpret_cast<uintptr_t>(B) & 31u) == 0 && ldb * es % 32 == 0;
    if (type == ElemType::kF32)
        w4_dequantize_kernel<float><<<grid, kDWarps * 32, 0, stream>>>(w, static_cast<float*>(B), ldb, vec);
    else if (type == ElemType::kBF16)
        w4_dequantize_kernel<__nv_bfloat16><<<grid, kDWarps * 32, 0, stream>>>(w, static_cast<__nv_bfloat16*>(B), ldb, vec);
    else
        w4_dequantize_kernel<__half><<<grid, kDWarps * 32, 0, stream>>>(w, static_cast<__half*>(B), ldb, vec);
    return cudaGetLastError();
}

cudaError_t launch_w4_gemm(const void* X, int64_t ldx, ElemType x_type, const void* codes,
                           const void* scales, void* C, int64_t ldc, ElemType c_type, int64_t M,
                           int64_t K, int64_t N, int group, int num_sms, cudaStream_t stream) {
    const W4 w = view(codes, scales, K, N, group);
    // the widest loads that every row of X allows, in bytes
    const uintptr_t bits = reinterpret_cast<uintptr_t>(X) | (M > 1 ? (uintptr_t)ldx * 2 : 0);
    const int align = (bits & 15u) == 0 ? 16 : (bits & 7u) == 0 ? 8 : (bits & 3u) == 0 ? 4 : 2;
    auto go = [&](auto x, auto c) {
        using T = decltype(x);
        using U = decltype(c);
        return launch_by_rows<T, U>(static_cast<const T*>(X), ldx, w, static_cast<U*>(C), ldc, M, align, num_sms, stream);
    };
    if (x_type == ElemType::kBF16)
        return c_type == ElemType::kF32 ? go(__nv_bfloat16(), float()) : go(__nv_bfloat16(), __nv_bfloat16());
    return c_type == ElemType::kF32 ? go(__half(), float()) : go(__half(), __half());
}

}  // namespace libgemm
