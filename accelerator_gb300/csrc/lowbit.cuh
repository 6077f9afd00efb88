// lowbit.cuh -- device helpers shared by the kernels on operands held in 4 or
// 8 bits: element types, the byte -> binary16 step, the warp-wide matrix
// instruction, and the lookup of a sequence by a row or a work unit.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <type_traits>

#include "debug.cuh"
#include "ptx.cuh"

namespace libgemm {

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
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma_16816<__nv_bfloat16>(float (&d)[4], uint32_t a0, uint32_t a1,
                                                         uint32_t a2, uint32_t a3, uint32_t b0,
                                                         uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same, binary16, from a C of its own.
__device__ __forceinline__ void mma_16816_from(float (&d)[4], const float* c, uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

constexpr uint64_t kWaitLimitNs = 2000000000ull;   // of any single wait

// A whole warp waits, and goes on or gives up together.  One lane looks (an
// arrival or a look by every lane is 32 operations on one word); a vote does not
// order memory, so what that lane saw reaches the others by the __syncwarp.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned* err) {
    const bool seen = __any_sync(0xFFFFFFFFu, threadIdx.x % 32 == 0 && mbar_wait(bar, parity, abort_flag, err, kWaitLimitNs));
    __syncwarp();
    return seen;
}
// Arrives once for a whole warp, after all its lanes' accesses.
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
    __syncwarp();
    if (threadIdx.x % 32 == 0) mbar_arrive(bar);
}

// Untiled bulk copy into this CTA's shared memory, completing on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// Waits for copies of this thread to land, whatever the other roles do.
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity, unsigned* err) {
    const uint64_t t0 = global_ns();
    while (!mbar_try_wait(bar, parity))
        if (global_ns() - t0 > kWaitLimitNs) {
            atomicOr(err, kErrTimeout);
            break;
        }
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

// Eight neighbours as the 16 or 32 bytes that hold them.
template <typename T>
struct Eight {
    uint4 v[sizeof(T) / 2];
    __device__ __forceinline__ float at(int i) const {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else if constexpr (std::is_same<T, __half>::value)
            return __half2float(__ushort_as_half((unsigned short)(w[i / 2] >> (16 * (i & 1)))));
        else return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    }
    __device__ __forceinline__ void put(int i, float y) {   // y one of the type's values, not of binary16
        uint32_t* w = reinterpret_cast<uint32_t*>(v);
        const uint32_t bits = __float_as_uint(y);
        if constexpr (sizeof(T) == 4) w[i] = bits;
        else w[i / 2] = i & 1 ? (w[i / 2] & 0xFFFFu) | (bits & 0xFFFF0000u) : (w[i / 2] & 0xFFFF0000u) | bits >> 16;
    }
};
template <typename T>
__device__ __forceinline__ Eight<T> load_eight(const T* p, bool vec) {
    Eight<T> e;
    if (vec) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) e.v[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
    } else if constexpr (sizeof(T) == 4) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = p[i];
        e.v[0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
        e.v[1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
    } else {
        const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
        uint32_t x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = (uint32_t)h[2 * i] | (uint32_t)h[2 * i + 1] << 16;
        e.v[0] = make_uint4(x[0], x[1], x[2], x[3]);
    }
    return e;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t c;
    asm("max.u16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
    return c;
}

// The largest magnitude of each of eight columns, as the bits of a float (from
// 0x7F800000 on: not finite); 16-bit types are compared two at a time.
template <typename T>
struct Tops {
    uint32_t m[sizeof(T) == 4 ? 8 : 4] = {};
    __device__ __forceinline__ void take(const Eight<T>& x) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(x.v);
#pragma unroll
        for (int i = 0; i < (sizeof(T) == 4 ? 8 : 4); ++i) {
            if constexpr (sizeof(T) == 4) m[i] = max(m[i], w[i] & 0x7FFFFFFFu);
            else m[i] = max_u16x2(m[i], w[i] & 0x7FFF7FFFu);
        }
    }
    __device__ __forceinline__ void across(int mask) {   // and of the lane that differs in `mask`
#pragma unroll
        for (int i = 0; i < (sizeof(T) == 4 ? 8 : 4); ++i) {
            const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, m[i], mask);
            if constexpr (sizeof(T) == 4) m[i] = max(m[i], o);
            else m[i] = max_u16x2(m[i], o);
        }
    }
    __device__ __forceinline__ uint32_t bits(int i) const {
        if constexpr (sizeof(T) == 4) return m[i];
        else if constexpr (std::is_same<T, __half>::value)
            return __float_as_uint(__half2float(__ushort_as_half((unsigned short)(m[i / 2] >> (16 * (i & 1))))));
        else return i & 1 ? m[i / 2] & 0xFFFF0000u : m[i / 2] << 16;
    }
    __device__ __forceinline__ uint32_t all() const {   // over the eight
        uint32_t t = 0;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i) t = max(t, m[i]);
            return t;
        } else {
            t = max_u16x2(max_u16x2(m[0], m[1]), max_u16x2(m[2], m[3]));
            Tops<T> one;
            one.m[0] = max(t & 0xFFFFu, t >> 16);
            return one.bits(0);
        }
    }
};

// The low bytes of four words.  An integer of a byte that is added to 1.5 *
// 2^23 is rounded there, ties to even, and left in the low byte.
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
__device__ __forceinline__ uint32_t low_bytes(float2 a, float2 b) {
    return low_bytes(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
}

// The largest b in [0, n) with value(b) <= x, for a non-decreasing value();
// 0 if there is none.  The lanes of a warp look at 32 places at once: a chain
// of two loads for a thousand sequences where halving has ten.
template <typename F>
__device__ __forceinline__ int last_not_above(int n, int64_t x, F value) {
    const int lane = threadIdx.x % 32;
    int lo = 0, hi = n;   // value(lo) <= x (or lo = 0), value(hi) > x (or hi = n)
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int64_t at = lo + (int64_t)lane * step;
        const unsigned below = __ballot_sync(0xFFFFFFFFu, at < hi && value((int)at) <= x);
        const int k = max(__popc(below) - 1, 0);
        lo += k * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// The same, where one guess is often right (one row for each sequence): a
// look at two places instead of the search.
template <typename F>
__device__ __forceinline__ int last_not_above(int n, int64_t x, int64_t guess, F value) {
    if (guess < n && value((int)guess) <= x && (guess + 1 == n || value((int)guess + 1) > x)) return (int)guess;
    return last_not_above(n, x, value);
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
    // Called by one CTA of a launch: reports offsets that do not ascend from 0 to `rows`.
    // A unit of the launch reports its own sequence's, but where offsets descend
    // a sequence may have no unit.
    __device__ __forceinline__ void check(unsigned* err) const {
        bool bad = false;
        for (int b = threadIdx.x; b < n; b += blockDim.x) bad |= !good(b);
        if (bad || (threadIdx.x == 0 && (__ldg(p) != 0 || __ldg(p + n) != rows))) atomicOr(err, kErrIndex);
    }
};

}  // namespace libgemm
