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
    __host__ __device__ int64_t nb() const { return (N + 15) / 16; }
};

// ---- quantise ----------------------------------------------------------------
// One CTA takes 128 rows x 64 columns (a whole number of groups and blocks):
// the tile goes through shared memory as floats, a thread finds the largest
// magnitude of 32 rows of one column, and each thread packs words of 8 codes.
constexpr int kQRows = 128, kQCols = 64, kQThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kQThreads)
    w4_quantize_kernel(const T* __restrict__ B, int64_t ldb, W4 w) {
    __shared__ float tile[kQRows][kQCols + 1];
    __shared__ uint32_t top[4][kQCols];
    __shared__ float scale[4][kQCols];
    const int64_t across = (w.N + kQCols - 1) / kQCols;
    const int64_t k0 = blockIdx.x / across * kQRows, n0 = blockIdx.x % across * kQCols;
    const int tid = threadIdx.x;
    [[maybe_unused]] const int64_t b_bytes = ((w.K - 1) * ldb + w.N) * (int64_t)sizeof(T);
    for (int i = tid; i < kQRows * kQCols; i += kQThreads) {
        const int r = i / kQCols, c = i % kQCols;
        const T* p = B + (k0 + r) * ldb + n0 + c;
        tile[r][c] = k0 + r < w.K && n0 + c < w.N && GEMM_DBG_OK(p, B, b_bytes, sizeof(T))
                         ? to_float(*p) : 0.0f;
    }
    __syncthreads();
    {
        const int c = tid % kQCols, part = tid / kQCols;
        uint32_t m = 0;   // magnitudes compare as their bits; above 0x7F800000 is NaN
        for (int r = 0; r < 32; ++r)
            m = max(m, __float_as_uint(tile[part * 32 + r][c]) & 0x7FFFFFFFu);
        top[part][c] = m;
    }
    __syncthreads();
    {
        const int c = tid % kQCols, part = tid / kQCols, per = w.group / 32;
        uint32_t m = 0;
        for (int i = 0; i < per; ++i) m = max(m, top[part / per * per + i][c]);
        const bool bad = m >= 0x7F800000u;
        const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(__uint_as_float(m), 7.0f));
        float s = __bfloat162float(sb);
        uint16_t bits = __bfloat16_as_ushort(sb);
        if (bad) s = 0.0f, bits = 0x7FC0;   // NaN; the codes are 0
        else if (s < kTiny) s = 0.0f, bits = 0;
        scale[part][c] = s;
        const int64_t g = (k0 + part * 32) / w.group, n = n0 + c;
        if (part % per == 0 && k0 + part * 32 < w.K && n < w.nb() * 16) {
            uint16_t* p = w.scales + ((n / 16 * w.groups + g) * 8 + n % 8) * 2 + n % 16 / 8;
            if (GEMM_DBG_OK(p, w.scales, w.nb() * w.groups * 32, 2)) *p = bits;
        }
    }
    __syncthreads();
    for (int i = tid; i < (kQRows / 64) * (kQCols / 16) * 128; i += kQThreads) {
        const int word = i % 128, kbl = i / 128 % (kQRows / 64), nbl = i / 128 / (kQRows / 64);
        const int lane = word / 4, j = word % 4, g = lane / 4, t = lane % 4;
        const int64_t nb = n0 / 16 + nbl, kb = k0 / 64 + kbl;
        if (nb >= w.nb() || kb >= w.kb) continue;
        uint32_t v = 0;
#pragma unroll
        for (int b = 0; b < 8; ++b) {
            const int hi = b & 1, e = (b >> 2) + 2 * ((b >> 1) & 1);
            const int r = kbl * 64 + 32 * (j >> 1) + 8 * t + 4 * (j & 1) + e, c = nbl * 16 + 8 * hi + g;
            const float s = scale[r / 32][c];
            const float q = s == 0.0f ? 0.0f : fminf(fmaxf(rintf(__fdiv_rn(tile[r][c], s)), -7.0f), 7.0f);
            v |= (uint32_t)((int)q + 8) << (4 * b);
        }
        uint32_t* p = w.codes + (nb * w.kb + kb) * 128 + word;
        if (GEMM_DBG_OK(p, w.codes, w.nb() * w.kb * 512, 4)) *p = v;
    }
}

// ---- dequantise --------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(kQThreads)
    w4_dequantize_kernel(W4 w, T* __restrict__ B, int64_t ldb) {
    __shared__ float tile[kQRows][kQCols + 1];
    const int64_t across = (w.N + kQCols - 1) / kQCols;
    const int64_t k0 = blockIdx.x / across * kQRows, n0 = blockIdx.x % across * kQCols;
    const int tid = threadIdx.x;
    for (int i = tid; i < (kQRows / 64) * (kQCols / 16) * 128; i += kQThreads) {
        const int word = i % 128, kbl = i / 128 % (kQRows / 64), nbl = i / 128 / (kQRows / 64);
        const int lane = word / 4, j = word % 4, g = lane / 4, t = lane % 4;
        const int64_t nb = n0 / 16 + nbl, kb = k0 / 64 + kbl;
        if (nb >= w.nb() || kb >= w.kb) continue;
        const uint32_t* p = w.codes + (nb * w.kb + kb) * 128 + word;
        if (!GEMM_DBG_OK(p, w.codes, w.nb() * w.kb * 512, 4)) continue;
        const uint32_t v = *p;
        const int64_t k = kb * 64 + 32 * (j >> 1);
        uint32_t s2 = 0;   // the scales of columns g and g + 8
        if (k < w.K) {
            const uint16_t* sp = w.scales + ((nb * w.groups + k / w.group) * 8 + g) * 2;
            if (GEMM_DBG_OK(sp, w.scales, w.nb() * w.groups * 32, 4)) s2 = *reinterpret_cast<const uint32_t*>(sp);
        }
#pragma unroll
        for (int b = 0; b < 8; ++b) {
            const int hi = b & 1, e = (b >> 2) + 2 * ((b >> 1) & 1);
            const float s = __uint_as_float(hi ? s2 & 0xFFFF0000u : s2 << 16);
            tile[kbl * 64 + 32 * (j >> 1) + 8 * t + 4 * (j & 1) + e][nbl * 16 + 8 * hi + g] =
                __fmul_rn((float)((int)((v >> (4 * b)) & 15u) - 8), s);
        }
    }
    __syncthreads();
    [[maybe_unused]] const int64_t b_bytes = ((w.K - 1) * ldb + w.N) * (int64_t)sizeof(T);
    for (int i = tid; i < kQRows * kQCols; i += kQThreads) {
        const int r = i / kQCols, c = i % kQCols;
        T* p = B + (k0 + r) * ldb + n0 + c;
        if (k0 + r < w.K && n0 + c < w.N && GEMM_DBG_OK(p, B, b_bytes, sizeof(T))) *p = from_float<T>(tile[r][c]);
    }
}

// ---- the product -------------------------------------------------------------
constexpr int kPWarps = 8;

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

// Eight neighbours x[k .. k + 7] of one row of X as four pairs; 0 past K.
template <typename T, bool VEC>
__device__ __forceinline__ uint4 load_x8(const T* row, int64_t k, int64_t K, bool live) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (!live || k >= K) return v;
    if (VEC && k + 8 <= K) return *reinterpret_cast<const uint4*>(row + k);
    uint32_t r[4] = {0, 0, 0, 0};
    const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
    for (int i = 0; i < 8; ++i)
        if (k + i < K) r[i / 2] |= (uint32_t)p[k + i] << (16 * (i & 1));
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// One CTA computes 16 columns of C for 8*MT rows: its warps take the blocks
// of 64 rows of W in turn and add their sums up at the end, in warp order.
template <typename T, typename U, int MT, bool VEC>
__global__ void __launch_bounds__(kPWarps * 32)
    w4_gemm_kernel(const T* __restrict__ X, int64_t ldx, W4 w, U* __restrict__ C, int64_t ldc,
                   int64_t M) {
    __shared__ float part[kPWarps][MT * 8][17];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int64_t nb = blockIdx.x % w.nb(), m0 = blockIdx.x / w.nb() * (8 * MT);
    [[maybe_unused]] const int64_t x_bytes = ((M - 1) * ldx + w.K) * (int64_t)sizeof(T);
    float total[MT][4] = {};
    const bool by_half = w.group == 32;   // scaled after each half block, or each block
    for (int kb = warp; kb < w.kb; kb += kPWarps) {
        const uint4* cp = reinterpret_cast<const uint4*>(w.codes + (nb * w.kb + kb) * 128) + lane;
        uint4 q = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
        if (GEMM_DBG_OK(cp, w.codes, w.nb() * w.kb * 512, 16)) q = __ldcs(cp);
        const uint32_t words[4] = {q.x, q.y, q.z, q.w};
        float acc[MT][4] = {};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t k = (int64_t)kb * 64 + 32 * h;
            uint32_t a0[4], a1[4];
            unpack8<T>(words[2 * h], a0);
            unpack8<T>(words[2 * h + 1], a1);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int64_t row = m0 + 8 * m + g;
                const uint4 x = load_x8<T, VEC>(X + row * ldx, k + 8 * t, w.K, row < M);
                mma_16816<T>(acc[m], a0[0], a0[1], a0[2], a0[3], x.x, x.y);
                mma_16816<T>(acc[m], a1[0], a1[1], a1[2], a1[3], x.z, x.w);
            }
            if (by_half || h == 1) {
                uint32_t s2 = 0;
                const int64_t kk = by_half ? k : (int64_t)kb * 64;
                if (kk < w.K) {
                    const uint16_t* sp = w.scales + ((nb * w.groups + kk / w.group) * 8 + g) * 2;
                    if (GEMM_DBG_OK(sp, w.scales, w.nb() * w.groups * 32, 4))
                        s2 = __ldg(reinterpret_cast<const uint32_t*>(sp));
                }
                const float lo = __uint_as_float(s2 << 16), hi = __uint_as_float(s2 & 0xFFFF0000u);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    total[m][0] = fmaf(acc[m][0], lo, total[m][0]);
                    total[m][1] = fmaf(acc[m][1], lo, total[m][1]);
                    total[m][2] = fmaf(acc[m][2], hi, total[m][2]);
                    total[m][3] = fmaf(acc[m][3], hi, total[m][3]);
                    acc[m][0] = acc[m][1] = acc[m][2] = acc[m][3] = 0.0f;
                }
            }
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        part[warp][8 * m + 2 * t][g] = total[m][0];
        part[warp][8 * m + 2 * t + 1][g] = total[m][1];
        part[warp][8 * m + 2 * t][g + 8] = total[m][2];
        part[warp][8 * m + 2 * t + 1][g + 8] = total[m][3];
    }
    __syncthreads();
    [[maybe_unused]] const int64_t c_bytes = ((M - 1) * ldc + w.N) * (int64_t)sizeof(U);
    for (int i = threadIdx.x; i < MT * 8 * 16; i += kPWarps * 32) {
        const int r = i / 16, c = i % 16;
        const int64_t row = m0 + r, col = nb * 16 + c;
        if (row >= M || col >= w.N) continue;
        float v = part[0][r][c];
#pragma unroll
        for (int p = 1; p < kPWarps; ++p) v += part[p][r][c];
        U* dst = C + row * ldc + col;
        if (GEMM_DBG_OK(dst, C, c_bytes, sizeof(U))) *dst = from_float<U>(v);
    }
}

W4 view(const void* codes, const void* scales, int64_t K, int64_t N, int group) {
    return W4{const_cast<uint32_t*>(static_cast<const uint32_t*>(codes)),
              const_cast<uint16_t*>(static_cast<const uint16_t*>(scales)), K, N, group,
              (int)((K + 63) / 64), (int)((K + group - 1) / group)};
}

template <typename T, typename U, bool VEC>
void launch_product(const T* X, int64_t ldx, const W4& w, U* C, int64_t ldc, int64_t M,
                    cudaStream_t stream) {
    const int mt = M <= 8 ? 1 : M <= 16 ? 2 : 4;
    const unsigned grid = (unsigned)(w.nb() * ((M + 8 * mt - 1) / (8 * mt)));
    if (mt == 1) w4_gemm_kernel<T, U, 1, VEC><<<grid, kPWarps * 32, 0, stream>>>(X, ldx, w, C, ldc, M);
    else if (mt == 2) w4_gemm_kernel<T, U, 2, VEC><<<grid, kPWarps * 32, 0, stream>>>(X, ldx, w, C, ldc, M);
    else w4_gemm_kernel<T, U, 4, VEC><<<grid, kPWarps * 32, 0, stream>>>(X, ldx, w, C, ldc, M);
}

}  // namespace

LIBGEMM_DEBUG_READER(w4_debug_flags)

cudaError_t launch_w4_quantize(const void* B, int64_t ldb, ElemType type, int64_t K, int64_t N,
                               int group, void* codes, void* scales, cudaStream_t stream) {
    const W4 w = view(codes, scales, K, N, group);
    const unsigned grid = (unsigned)(((K + kQRows - 1) / kQRows) * ((N + kQCols - 1) / kQCols));
    if (type == ElemType::kF32)
        w4_quantize_kernel<float><<<grid, kQThreads, 0, stream>>>(static_cast<const float*>(B), ldb, w);
    else if (type == ElemType::kBF16)
        w4_quantize_kernel<__nv_bfloat16><<<grid, kQThreads, 0, stream>>>(static_cast<const __nv_bfloat16*>(B), ldb, w);
    else
        w4_quantize_kernel<__half><<<grid, kQThreads, 0, stream>>>(static_cast<const __half*>(B), ldb, w);
    return cudaGetLastError();
}

cudaError_t launch_w4_dequantize(const void* codes, const void* scales, int64_t K, int64_t N,
                                 int group, void* B, int64_t ldb, ElemType type,
                                 cudaStream_t stream) {
    const W4 w = view(codes, scales, K, N, group);
    const unsigned grid = (unsigned)(((K + kQRows - 1) / kQRows) * ((N + kQCols - 1) / kQCols));
    if (type == ElemType::kF32)
        w4_dequantize_kernel<float><<<grid, kQThreads, 0, stream>>>(w, static_cast<float*>(B), ldb);
    else if (type == ElemType::kBF16)
        w4_dequantize_kernel<__nv_bfloat16><<<grid, kQThreads, 0, stream>>>(w, static_cast<__nv_bfloat16*>(B), ldb);
    else
        w4_dequantize_kernel<__half><<<grid, kQThreads, 0, stream>>>(w, static_cast<__half*>(B), ldb);
    return cudaGetLastError();
}

cudaError_t launch_w4_gemm(const void* X, int64_t ldx, ElemType x_type, const void* codes,
                           const void* scales, void* C, int64_t ldc, ElemType c_type, int64_t M,
                           int64_t K, int64_t N, int group, cudaStream_t stream) {
    const W4 w = view(codes, scales, K, N, group);
    const bool vec = (reinterpret_cast<uintptr_t>(X) & 15u) == 0 && (ldx % 8 == 0 || M == 1);
    auto go = [&](auto x, auto c) {
        using T = decltype(x);
        using U = decltype(c);
        if (vec) launch_product<T, U, true>(static_cast<const T*>(X), ldx, w, static_cast<U*>(C), ldc, M, stream);
        else launch_product<T, U, false>(static_cast<const T*>(X), ldx, w, static_cast<U*>(C), ldc, M, stream);
    };
    if (x_type == ElemType::kBF16) {
        if (c_type == ElemType::kF32) go(__nv_bfloat16(), float());
        else go(__nv_bfloat16(), __nv_bfloat16());
    } else {
        if (c_type == ElemType::kF32) go(__half(), float());
        else go(__half(), __half());
    }
    return cudaGetLastError();
}

}  // namespace libgemm
