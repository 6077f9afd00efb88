// lowbit.cuh -- device helpers shared by the kernels on operands held in 4 or
// 8 bits: element types, the byte -> binary16 step, the warp-wide matrix
// instruction, and the lookup of a sequence by a row or a work unit.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "debug.cuh"
#include "ptx.cuh"

namespace libgemm {

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_float<__half>(__half x) { return __half2float(x); }

// Rounded once, to nearest, ties to even.
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// D (16 x 8, fp32) += A (16 x 16) * B (16 x 8), warp-wide.  With g = lane / 4
// and t = lane % 4: a[0], a[2] are row g, a[1], a[3] row g + 8, k = 2t, 2t + 1
// in a[0], a[1] and 2t + 8, 2t + 9 in a[2], a[3]; b[0], b[1] the same k of
// column g; d[0], d[1] are row g, columns 2t, 2t + 1, d[2], d[3] row g + 8.
template <typename T>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma_16816<__half>(float (&d)[4], uint32_t a0, uint32_t a1,
                                                  uint32_t a2, uint32_t a3, uint32_t b0,
                                                  uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma_16816<__nv_bfloat16>(float (&d)[4], uint32_t a0, uint32_t a1,
                                                         uint32_t a2, uint32_t a3, uint32_t b0,
                                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two code bytes u = c + 128 beside a byte 0x64 each are the binary16 values
// 1024 + u; less 1152 they are c, exactly.
__device__ __forceinline__ uint32_t halves_from_biased(uint32_t x) {
    const uint32_t bias = 0x64806480u;   // 1152, twice
    const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&bias));
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t codes01(uint32_t w) { return halves_from_biased(__byte_perm(w, 0x64646464u, 0x4140)); }
__device__ __forceinline__ uint32_t codes23(uint32_t w) { return halves_from_biased(__byte_perm(w, 0x64646464u, 0x4342)); }

// The largest b in [0, n) with value(b) <= x, for a non-decreasing value();
// 0 if there is none.
template <typename F>
__device__ __forceinline__ int last_not_above(int n, int64_t x, F value) {
    int lo = 0, hi = n;   // value(lo) <= x (or lo = 0), value(hi) > x (or hi = n)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (value(mid) <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// A batch's row offsets as the caller gave them: sequence b has rows [at(b),
// at(b + 1)).  Offsets outside [0, rows] or descending are reported and read
// as an empty sequence.
struct Starts {
    const int32_t* p;
    int n;         // sequences
    int64_t rows;
    __device__ __forceinline__ int64_t at(int b) const {
        if (!GEMM_DBG_OK(p + b, p, (n + 1) * (int64_t)4, 4)) return 0;
        const int64_t v = __ldg(p + b);
        return v < 0 ? 0 : v > rows ? rows : v;
    }
    __device__ __forceinline__ bool good(int b) const {
        const int64_t s = __ldg(p + b), e = __ldg(p + b + 1);
        return s >= 0 && s <= e && e <= rows;
    }
};

}  // namespace libgemm
