// kv_prompt.cu -- attention of many query rows (prompts) over a paged cache of 8
// or 4 bits, on the 5th-generation tensor cores.
//
// One CTA takes 256 query rows of a sequence and cache head -- two tiles of
// 128, so that what is done to the keys and values of a block of 128 tokens
// serves both -- and walks the tokens.  Its warps have fixed roles:
//   warps 0-3, 4-7  softmax of tile 0 and tile 1, one thread a row: scores
//       from tensor memory, weights back as binary16 over the scores, and the
//       sums so far rescaled in tensor memory when a maximum is passed;
//   warps 8-11  the cache: codes of a block from where the copies put them, as
//       binary16 integers (exact) in the 128-byte swizzle that the matrix unit
//       reads; the keys with d, the values with the token as the reduced
//       dimension, from the same layout;
//   warp 12  one thread issues tcgen05.mma: S_i = Q_i K^T (both from shared
//       memory), O_i += P_i V (P from tensor memory);
//   warp 13  looks the pages up and copies their codes in bulk.
// The two tiles are half a step apart: while one tile's softmax runs, the
// matrix unit works for the other.  Tensor memory holds S_0, S_1 (128 columns
// each, P over the first half of its S) and O_0, O_1: all of its 512 columns.
//
// A block of 128 tokens and 256 rows has to take 2048 cycles of the matrix unit
// and 2500 of shared memory (operands, and the codes' way into them); it took
// about 5400 when traced, the length of one tile's chain: scores 880, their way to the
// softmax 480, load and maximum 600, exponentials and weights 1250, their way
// back 430, output 740.  The tensor pipe's counter is active for 30 % of the
// cycles.  4 x 1000 rows of 32 heads over up to 8192 tokens of 8: 418 us, 617
// TFLOP/s; a second maximum a row (see `mv`) and what orders a warp behind its
// waits are 6 us of it.  Measured and left, when it took 412 us: scores loaded and
// weighed 32 at a time (593 us), weights against the previous maximum in one pass
// (524 us), scores of 64 tokens in two buffers a tile, so that the next are ready
// early (511 us: a product 64 wide takes the matrix unit as long as one 128 wide,
// 515 cycles).
//
// 4 bits.  A token's keys and values have scales of their own, and a code times its
// scale, c in [-7, 7] times 8 bits, is exact in binary16's 11.  So the copying warp
// brings the scales of 16 tokens to one power of two, S in [2^15, 2^16) for the
// largest, as binary16, the cache's warps make c * S * 2^-24 of the codes, and what
// stands outside of the products is a power of two alone, where the 8-bit cache has
// its page's scale.  A masked nibble is the number u * 2^-24 (or 2^-20), below
// binary16's normal range, so that c * S * 2^-24 is one fused multiply-add, exact
// for scales down to 2^-8 of the largest; blocks that have others take c * S * 2^-4
// by a subtraction and a product, exact down to 2^-28.  Codes wait in two buffers.
// Scales of tokens that no row of the tile sees are taken for 0; a token that reads
// as NaN gets keys of NaN, which make NaN of the scores of the rows that see it, and
// values of 0.  Sums on tensor memory are truncated, 16 tokens at a time: of values all of
// one sign results are low by 3e-4 of themselves over 65536 tokens and 9e-4 over 200001,
// over either cache; of values of both signs by no more than the rounding of binary16.
// The example above takes 468 us over 4 bits, 550 TFLOP/s, and 402 with
// the arithmetic on the codes left out: the chain of a tile, as above, then the cache's
// warps.  One buffer of codes and a product after a subtraction for all blocks took
// 499 us, NaN looked for with each score 585 (registers spilled).
//
// Every wait is bounded; a role that gives up raises the abort flag, all stop,
// and the matrix unit is drained before tensor memory is freed.
#include "kv_attention.cuh"

namespace libgemm {
namespace {

constexpr int kTile = 128, kRows = 2 * kTile, kStep = 128;   // rows of a tile and a CTA, tokens of a block
constexpr int kSub = 16, kSubs = kStep / kSub;               // tokens that share a page for certain
// Code buffers of each operand, and blocks whose page data are kept.
constexpr int code_buffers(int bits) { return bits == 4 ? 2 : 1; }
constexpr int kept_blocks(int bits) { return bits == 4 ? 5 : 4; }
constexpr int kSoftWarps = 8, kCacheWarps = 4, kThreads = (kSoftWarps + kCacheWarps + 4) * 32;
// Registers of a thread: launched with 128, then shared out among the roles
// (whole warpgroups), whose sum is that of the launch.  Of 4 bits the copying warp
// also looks after scales.
constexpr int kLaunchRegs = 128, kSoftRegs = 184;
constexpr int cache_regs(int bits) { return bits == 8 ? 104 : 88; }
constexpr int issue_regs(int bits) { return bits == 8 ? 40 : 56; }
static_assert(kSoftRegs * kSoftWarps + cache_regs(8) * kCacheWarps + issue_regs(8) * 4 <= kLaunchRegs * kThreads / 32, "");
static_assert(kSoftRegs * kSoftWarps + cache_regs(4) * kCacheWarps + issue_regs(4) * 4 <= kLaunchRegs * kThreads / 32, "");
constexpr int kSlab = kTile * 128;                           // 128 rows of 64 binary16

// What a softmax thread needs of 16 tokens: the key scale, log2 of the
// value scale (-inf for one of 0).
struct alignas(16) PageData {
    float ks, log_v;
    uint32_t plain;      // 1: there, and reads as numbers; 0: reads as NaN; 2: not there
};

template <int D, int BITS>
struct Smem {
    static constexpr int kOperand = D / 64 * kSlab;          // 128 x D binary16
    static constexpr int kQ = 0, kK = 2 * kOperand, kV = kK + 2 * kOperand;
    static constexpr int kCodeBytes = kStep * D * BITS / 8;  // keys' and values' each
    static constexpr int kBuffers = code_buffers(BITS), kSlots = kept_blocks(BITS);
    // codes [buffer][keys, values]; of 4 bits binary16 scales, and whether they are far apart, likewise
    static constexpr int kCodes = kV + 2 * kOperand, kScales = kCodes + 2 * kBuffers * kCodeBytes;
    static constexpr int kWide = kScales + (BITS == 4 ? 2 * kBuffers * kStep * 2 : 0), kInfo = kWide + (BITS == 4 ? 16 : 0);
    static constexpr int kBars = kInfo + kSlots * kSubs * (int)sizeof(PageData);
    static constexpr int kBytes = kBars + 208 + 1024;        // and the alignment
    static_assert(kBytes + 16 <= 227 * 1024, "");
};
// Barriers: keys and values full / empty (two buffers), per tile scores full,
// weights full (of the first and of the last 64 tokens), output done; codes
// full / empty (keys, values; buffers); the drain.
enum { kKFull = 0, kKEmpty = 2, kVFull = 4, kVEmpty = 6, kSFull = 8, kPFull = 10, kODone = 14, kCFull = 16, kCEmpty = 20, kDrain = 24 };

__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
        "}\n" ::"r"(d), "r"(a), "l"(bdesc), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]),
        "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
        "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_ld_x16(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
// Waits for the tensor memory loads; nothing that reads r moves before it.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
    asm volatile("" : "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                      "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}
template <int N>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Chunk c (eight binary16) of row r of a 64-wide slab: 128-byte swizzle.
__device__ __forceinline__ uint32_t swizzled(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

// What makes values of a word's codes: of a pair of scales S, c * S * 2^-24, or with
// WIDE c * S * 2^-4.
__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
__device__ __forceinline__ uint32_t bits_of(__half2 x) { return *reinterpret_cast<const uint32_t*>(&x); }
struct Factors {
    bool wide;
    __half2 low, high, less;
    __device__ __forceinline__ Factors(uint32_t scales, bool w) : wide(w) {
        const __half2 s = as_half2(scales), sixteenth = as_half2(0x2C002C00u);
        high = __hmul2(s, sixteenth);
        low = wide ? high : s;
        less = __hmul2(s, as_half2(0x80088008u));   // -8 * 2^-24
    }
    // The nibbles of bits 0-3 and 16-19, 4-7 and 20-23, 8-11 and 24-27, and the last ones.
    __device__ __forceinline__ void four(uint32_t x, uint32_t (&d)[4]) const {
        const uint32_t y = x >> 8, w[4] = {x & 0x000F000Fu, x & 0x00F000F0u, y & 0x000F000Fu, y & 0x00F000F0u};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!wide) d[i] = bits_of(__hfma2(as_half2(w[i]), i & 1 ? high : low, less));
            else if (i & 1) d[i] = bits_of(__hmul2(__hsub2(as_half2(w[i] | 0x54005400u), as_half2(0x54805480u)), low));   // 64 + u
            else d[i] = bits_of(__hmul2(__hsub2(as_half2(w[i] | 0x64006400u), as_half2(0x64086408u)), low));              // 1024 + u
        }
    }
};
template <typename F>
__device__ __forceinline__ void with_values(uint32_t wide, F f) {
    if (wide) f(std::true_type());
    else f(std::false_type());
}

template <typename T, int D, int BITS>
__global__ void __launch_bounds__(kThreads, 1) kv_prompt_kernel(const AttnArgs a, bool o_vec) {
    using L = Smem<D, BITS>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    PageData* info = reinterpret_cast<PageData*>(smem + L::kInfo);
    const uint32_t bars = base + L::kBars;
    volatile int* abort_flag = &s_abort;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    constexpr int kSlots = L::kSlots;
    // The barriers of block j's codes, and the phase in which they are its.
    auto code_bar = [&](int which, int values, int j) { return bars + 8 * (which + values * L::kBuffers + j % L::kBuffers); };
    auto code_parity = [&](int j) { return (uint32_t)(j / L::kBuffers) & 1u; };
    // Heads fastest: sequences come one after another, long ones seldom last.
    const int h = blockIdx.x % a.c.heads, split = blockIdx.x / a.c.heads % a.splits, u = blockIdx.x / a.c.heads / a.splits;
    Tile tile;
    if (!tile.find(a, u, kRows, kStep, h == 0 && split == 0) || split >= tile.active) return;
    grid_launch_dependents();   // a joining launch may start its set-up
    const int begin = split * tile.per, blocks = min(tile.steps, begin + tile.per) - begin;
    const int tok_begin = tile.tok0 + begin * kStep;
    const int tiles = tile.r0 + kTile < tile.nrows ? 2 : 1;
    const int32_t* table = a.b.table + tile.seq * a.b.width;
    const int log2 = a.c.page_log2;

    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(bars + 8 * (kKFull + i), kCacheWarps);
            mbar_init(bars + 8 * (kVFull + i), kCacheWarps);
            mbar_init(bars + 8 * (kKEmpty + i), 1);
            mbar_init(bars + 8 * (kVEmpty + i), 1);
            mbar_init(bars + 8 * (kSFull + i), 2);   // the matrix unit, and its issuer for the page data
            mbar_init(bars + 8 * (kPFull + 2 * i), kTile / 32);
            mbar_init(bars + 8 * (kPFull + 2 * i + 1), kTile / 32);
            mbar_init(bars + 8 * (kODone + i), 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(bars + 8 * (kCFull + i), 1);
            mbar_init(bars + 8 * (kCEmpty + i), kCacheWarps);
        }
        mbar_init(bars + 8 * kDrain, 1);
        mbar_fence_init();
    }
    if (warp == kSoftWarps + kCacheWarps) {
        tmem_alloc(smem_u32(&s_tmem), 512);
        tmem_relinquish();
    }
    // The softmax threads bring their row of Q to shared memory (as binary16;
    // bfloat16 rows brought to [1, 2) by a power of two, exact but for elements
    // under 2^-14 of the row's largest).
    float row_scale = 0.0f;
    const int in_tile = threadIdx.x % kTile, which = threadIdx.x / kTile;   // for softmax threads
    const int my_row = tile.r0 + threadIdx.x;
    if (warp < kSoftWarps) {
        const bool live = my_row < tile.nrows;
        [[maybe_unused]] const int64_t q_bytes =
            ((a.b.rows - 1) * a.Q.row + (a.q_heads - 1) * a.Q.head + D) * (int64_t)sizeof(T);
        const unsigned r = live ? my_row : 0;
        const T* p = static_cast<const T*>(a.Q.p) + (int64_t)(tile.row0 + r / a.share) * a.Q.row + (int64_t)(h * a.share + r % a.share) * a.Q.head;
        float up = 1.0f, down = 1.0f;
        if constexpr (!std::is_same<T, __half>::value) {
            float top = 0.0f;
            for (int c = 0; c < D / 8; ++c) {
                Eight<T> x = {};
                if (live && GEMM_DBG_OK(p + 8 * c, a.Q.p, q_bytes, 16)) x = load_eight(p + 8 * c, a.q_vec);
#pragma unroll
                for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x.at(e)));
            }
            const int e = (int)(__float_as_uint(top) >> 23);   // biased exponent
            if (top > 0.0f && top < INFINITY) {
                const int k = max(1, min(253, e));
                up = __uint_as_float((uint32_t)k << 23);             // 2^(k - 127)
                down = __uint_as_float((uint32_t)(254 - k) << 23);   // 2^(127 - k)
            }
        }
        row_scale = fabsf(a.scale_log2) * up;
        if (a.scale_log2 < 0.0f) down = -down;
        const uint32_t q0 = base + L::kQ + which * L::kOperand;
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
            Eight<T> x = {};
            if (live && GEMM_DBG_OK(p + 8 * c, a.Q.p, q_bytes, 16)) x = load_eight(p + 8 * c, a.q_vec);
            // in the order in which a chunk has the keys' elements: of 4 bits e beside e + 4
            constexpr int kMate = BITS == 4 ? 4 : 1, kNext = BITS == 4 ? 1 : 2;
            auto two = [&](int i) { return pack2<__half>(x.at(kNext * i) * down, x.at(kNext * i + kMate) * down); };
            st_shared_v4(q0 + c / 8 * kSlab + swizzled(in_tile, c % 8), two(0), two(1), two(2), two(3));
        }
        fence_proxy_async_shared();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;

    if (warp >= kSoftWarps && warp < kSoftWarps + kCacheWarps) {
        // ---------------- the cache ----------------
        fewer_registers<cache_regs(BITS)>();
        // 8 bits: lanes of a token, 16 codes each; 4 bits: pieces of D / 8 bytes, of a
        // token's keys and of two tokens' values.
        constexpr int kLanes = BITS == 8 ? D / 16 : 4, kWords = D / 32;
        constexpr int kPassRows = kCacheWarps * 32 / kLanes, kPasses = kStep / kPassRows;
        const int ct = threadIdx.x - kSoftWarps * 32;
        // A quarter of a warp holds halves of two rows, neighbours or (4 bits) four
        // apart: its 16-byte stores then meet all eight chunk positions of the swizzle.
        const int piece = D == 128 && BITS == 8 ? ct % 4 + 4 * (ct / 8 % 2) : ct % 4;
        const int sub_row = BITS == 4 ? ct / 32 * 8 + ct / 8 % 4 + 4 * (ct / 4 % 2) : D == 128 ? ct / 16 * 2 + ct / 4 % 2 : ct / 4;
        uint4 w[BITS == 8 ? kPasses : 1];
        uint32_t words[BITS == 4 ? kPasses : 1][kWords], scales[BITS == 4 ? kPasses : 1], wide = 0;
        auto get = [&](int values, int j) {
            if (!warp_wait(code_bar(kCFull, values, j), code_parity(j), abort_flag, a.err)) return false;
            const int buffer = j % L::kBuffers * 2 + values;
            const uint32_t codes = base + L::kCodes + buffer * L::kCodeBytes;
            if constexpr (BITS == 8) {
                const uint32_t from = codes + sub_row * D + 16 * piece;
#pragma unroll
                for (int i = 0; i < kPasses; ++i) w[i] = lds128(from + i * kPassRows * D);
            } else {
                const uint32_t at = base + L::kScales + buffer * (2 * kStep);
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(wide) : "r"(base + L::kWide + 4 * buffer));
#pragma unroll
                for (int i = 0; i < kPasses; ++i) {
                    // values: warp by warp the eights of tokens, of which a lane has a pair
                    const int row = sub_row + i * kPassRows, eight = i * kCacheWarps + ct / 32;
                    const uint32_t from = codes + (values ? eight * (4 * D) + ct % 32 * (D / 8) : row * (D / 2) + piece * (D / 8));
                    if constexpr (D == 128) {
                        const uint4 v = lds128(from);
                        words[i][0] = v.x, words[i][1] = v.y, words[i][2] = v.z, words[i][3] = v.w;
                    } else {
                        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(words[i][0]), "=r"(words[i][1]) : "r"(from));
                    }
                    if (values) {
                        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(scales[i]) : "r"(at + 2 * (8 * eight + 2 * (ct % 4))));
                    } else {
                        uint16_t one;
                        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(one) : "r"(at + 2 * row));
                        scales[i] = (uint32_t)one * 0x10001u;
                    }
                }
            }
            return true;
        };
        auto put = [&](int values, uint32_t to) {
            if constexpr (BITS == 8) {
                const int c = 2 * piece % 8;
                const uint32_t at = to + 2 * piece / 8 * kSlab + sub_row * 128, r = sub_row & 7;
#pragma unroll
                for (int i = 0; i < kPasses; ++i) {
                    const uint32_t row = at + i * kPassRows * 128;
                    st_shared_v4(row + ((c ^ r) << 4), codes01(w[i].x), codes23(w[i].x), codes01(w[i].y), codes23(w[i].y));
                    st_shared_v4(row + (((c + 1) ^ r) << 4), codes01(w[i].z), codes23(w[i].z), codes01(w[i].w), codes23(w[i].w));
                }
            } else if (!values) {   // word e is the chunk of elements 32 e + 8 piece on
                const uint32_t at = to + sub_row * 128, r = sub_row & 7;
                with_values(wide, [&](auto values_of) {
#pragma unroll
                    for (int i = 0; i < kPasses; ++i) {
                        const Factors f(scales[i], decltype(values_of)::value);
#pragma unroll
                        for (int e = 0; e < kWords; ++e) {
                            uint32_t d[4];
                            f.four(words[i][e], d);
                            st_shared_v4(at + e / 2 * kSlab + i * kPassRows * 128 + (((4 * (e % 2) + piece) ^ r) << 4), d[0], d[1], d[2], d[3]);
                        }
                    }
                });
            } else {                // words 2e, 2e + 1 are four elements each of two tokens, chunk g of slab e
                const int g = ct % 32 / 4, t = ct % 4;
                with_values(wide, [&](auto values_of) {
#pragma unroll
                    for (int i = 0; i < kPasses; ++i) {
                        const uint32_t at = to + (8 * (i * kCacheWarps + ct / 32) + 2 * t) * 128;
                        const Factors f(scales[i], decltype(values_of)::value);
#pragma unroll
                        for (int e = 0; e < D / 64; ++e) {
                            uint32_t even[4], odd[4];
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                uint32_t d[4];
                                f.four(words[i][2 * e + q], d);
                                even[2 * q] = __byte_perm(d[0], d[1], 0x5410), even[2 * q + 1] = __byte_perm(d[2], d[3], 0x5410);
                                odd[2 * q] = __byte_perm(d[0], d[1], 0x7632), odd[2 * q + 1] = __byte_perm(d[2], d[3], 0x7632);
                            }
                            st_shared_v4(at + e * kSlab + ((g ^ (2 * t)) << 4), even[0], even[1], even[2], even[3]);
                            st_shared_v4(at + e * kSlab + 128 + ((g ^ (2 * t + 1)) << 4), odd[0], odd[1], odd[2], odd[3]);
                        }
                    }
                });
            }
            fence_proxy_async_shared();
        };
        for (int j = 0; j < blocks; ++j) {
            const int buf = j & 1;
            const uint32_t parity = (uint32_t)(j >> 1) & 1u;
            if (!get(0, j)) break;
            warp_arrive(code_bar(kCEmpty, 0, j));
            if (!warp_wait(bars + 8 * (kKEmpty + buf), parity ^ 1u, abort_flag, a.err)) break;
            put(0, base + L::kK + buf * L::kOperand);
            warp_arrive(bars + 8 * (kKFull + buf));
            if (!get(1, j)) break;
            warp_arrive(code_bar(kCEmpty, 1, j));
            if (!warp_wait(bars + 8 * (kVEmpty + buf), parity ^ 1u, abort_flag, a.err)) break;
            put(1, base + L::kV + buf * L::kOperand);
            warp_arrive(bars + 8 * (kVFull + buf));
        }
    } else if (warp >= kSoftWarps + kCacheWarps) {
        // ---------------- the matrix unit ----------------
        fewer_registers<issue_regs(BITS)>();
        if (threadIdx.x == (kSoftWarps + kCacheWarps) * 32) {
            constexpr uint32_t kIdS = make_idesc(0, kTile, kStep, false, false), kIdO = make_idesc(0, kTile, D, false, true);
            auto scores = [&](int i, int buf) {   // S_i = Q_i K^T
                const uint32_t q = base + L::kQ + i * L::kOperand, k = base + L::kK + buf * L::kOperand;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    tc_mma<TcKind::kF16>(tmem + i * kStep, smem_desc_sw128(q + kk / 4 * kSlab + kk % 4 * 32, 16, 1024),
                                         smem_desc_sw128(k + kk / 4 * kSlab + kk % 4 * 32, 16, 1024), kIdS, kk != 0);
                tc_commit(bars + 8 * (kSFull + i));
                mbar_arrive(bars + 8 * (kSFull + i));
            };
            bool ok = blocks > 0 && mbar_wait(bars + 8 * kKFull, 0, abort_flag, a.err, kWaitLimitNs);
            if (ok) {
                tc_fence_after();
                for (int i = 0; i < tiles; ++i) scores(i, 0);
                tc_commit(bars + 8 * kKEmpty);
            }
            for (int j = 0; ok && j < blocks; ++j) {
                const int buf = j & 1;
                ok = mbar_wait(bars + 8 * (kVFull + buf), (uint32_t)(j >> 1) & 1u, abort_flag, a.err, kWaitLimitNs);
                for (int i = 0; ok && i < tiles; ++i) {
                    const uint32_t v = base + L::kV + buf * L::kOperand;
                    // O_i += P_i V, each half as soon as its weights are there
                    for (int half = 0; ok && half < 2; ++half) {
                        if (!(ok = mbar_wait(bars + 8 * (kPFull + 2 * i + half), (uint32_t)j & 1u, abort_flag, a.err, kWaitLimitNs))) break;
                        tc_fence_after();
#pragma unroll
                        for (int k = 0; k < kStep / 32; ++k) {
                            const int kk = half * (kStep / 32) + k;
                            tc_mma_ts(tmem + 2 * kStep + i * kStep, tmem + i * kStep + kk * 8,
                                      smem_desc_sw128(v + kk * 16 * 128, kSlab, 1024), kIdO, (j | kk) != 0);
                        }
                    }
                    if (!ok) break;
                    tc_commit(bars + 8 * (kODone + i));
                    if (i == tiles - 1) tc_commit(bars + 8 * (kVEmpty + buf));
                    if (j + 1 < blocks) {
                        if (i == 0 && !(ok = mbar_wait(bars + 8 * (kKFull + (buf ^ 1)), (uint32_t)((j + 1) >> 1) & 1u, abort_flag, a.err, kWaitLimitNs))) break;
                        tc_fence_after();
                        scores(i, buf ^ 1);
                        if (i == tiles - 1) tc_commit(bars + 8 * (kKEmpty + (buf ^ 1)));
                    }
                }
            }
            // Everything issued is done before tensor memory is freed.
            tc_commit(bars + 8 * kDrain);
            drain(bars + 8 * kDrain, 0, a.err);
        }
        if (warp == kSoftWarps + kCacheWarps + 1) {
            // ---------------- the copies: lane i < 8 looks after 16 tokens of a block,
            // of 4 bits lane i after 4, whose scales it brings down ----------------
            constexpr int kTokens = BITS == 8 ? kSub : 4;
            [[maybe_unused]] const int64_t code_bytes = a.c.pages * a.c.heads * ((int64_t)D << log2);
            [[maybe_unused]] const int64_t extent = a.c.pages * a.c.heads * a.c.record();
            const int chunk = min(kStep, 1 << log2);   // tokens of one copy
            struct Sub { int64_t from; float ks, vs; bool live; uint2 scales[BITS == 4 ? 2 : 1]; };
            auto look = [&](int j) {
                Sub s{0, 0.0f, 0.0f, false, {}};
                const int tok = tok_begin + j * kStep + lane * kTokens;
                if (lane * kTokens < kStep && j < blocks && tile.page_seen(tok, log2)) {
                    const int64_t page = __ldg(table + (tok >> log2));
                    s.live = page >= 0 && page < a.c.pages;
                    if (!s.live) atomicOr(a.err, kErrIndex);
                    else if constexpr (BITS == 4) {
                        s.from = (page * a.c.heads + h) * a.c.record();   // of the page
                        const uint8_t* at = a.c.data + s.from + (D << log2) + 2 * (tok & ((1 << log2) - 1));
                        if (GEMM_DBG_OK(at, a.c.data, extent, 8)) s.scales[0] = __ldg(reinterpret_cast<const uint2*>(at));
                        at += 2 << log2;
                        if (GEMM_DBG_OK(at, a.c.data, extent, 8)) s.scales[1] = __ldg(reinterpret_cast<const uint2*>(at));
                    } else {
                        const int64_t ph = page * a.c.heads + h;
                        s.from = ((ph << log2) + (tok & ((1 << log2) - 1))) * D;
                        s.ks = __ldg(a.c.ks + ph);
                        s.vs = __ldg(a.c.vs + ph);
                    }
                }
                return s;
            };
            Sub now = look(0);
            int issued[2] = {0, 0};
            for (int j = 0; j < blocks; ++j) {
                const Sub next = look(j + 1);
                // the first tokens of a page's part fetch all of it
                bool copies = now.live && lane * kTokens % chunk == 0;
                if constexpr (BITS == 8) {
                    if (copies) copies = GEMM_DBG_OK(a.c.k + now.from, a.c.k, code_bytes, chunk * D) && GEMM_DBG_OK(a.c.v + now.from, a.c.v, code_bytes, chunk * D);
                } else {
                    if (copies) copies = GEMM_DBG_OK(a.c.data + now.from, a.c.data, extent, chunk * D);
                }
                const uint32_t part = (uint32_t)(chunk * D * BITS / 8), bytes = (uint32_t)__popc(__ballot_sync(0xFFFFFFFFu, copies)) * part;
                // 4 bits: of both operands, this lane's scales as binary16 times 2^(142 - e),
                // e the biased exponent of the largest of 16 tokens' (held so that the power
                // of two is normal); whether any of the block's is far from that
                uint32_t held[2][2] = {}, unit[2] = {}, wide[2] = {};
                bool zero[2] = {};
                if constexpr (BITS == 4) {
                    const int tok = tok_begin + j * kStep + lane * kTokens;
                    uint32_t bits[2][4], nan = 0;
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        bits[v][0] = now.scales[v].x & 0x7FFFu, bits[v][1] = now.scales[v].x >> 16 & 0x7FFFu;
                        bits[v][2] = now.scales[v].y & 0x7FFFu, bits[v][3] = now.scales[v].y >> 16 & 0x7FFFu;
                        uint32_t most = 0;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (!now.live || tok + i < tile.lo || tok + i >= tile.hi) bits[v][i] = 0;
                            if (bits[v][i] >= 0x7F80u) nan |= 1u << i, bits[v][i] = 0;
                            most = max(most, bits[v][i]);
                        }
                        most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
                        most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
                        unit[v] = max(most >> 7, 15u);
                        zero[v] = most == 0;
                        bool far = unit[v] > 245u;   // (2^(e - 118) is normal)
#pragma unroll
                        for (int i = 0; i < 4; ++i) far |= bits[v][i] != 0 && (bits[v][i] >> 7) + 8 < unit[v];
                        wide[v] = __any_sync(0xFFFFFFFFu, far);
                    }
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        const float by = __uint_as_float((269u - unit[v]) << 23);
                        float s[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            s[i] = __uint_as_float(bits[v][i] << 16) * by;
                            if (nan >> i & 1u) s[i] = v ? 0.0f : __uint_as_float(0x7FC00000u);
                        }
                        held[v][0] = pack2<__half>(s[0], s[1]);
                        held[v][1] = pack2<__half>(s[2], s[3]);
                    }
                }
                bool ok = true;
#pragma unroll
                for (int values = 0; values < 2; ++values) {
                    // Page data of block j go where those of block j - 4 were: its keys' turn
                    // comes when the keys of j - 1 are taken, so the values of j - 4 are used up
                    // (4 bits: of j - 5, j - 2 and j - 5).
                    if (!(ok = warp_wait(code_bar(kCEmpty, values, j), code_parity(j) ^ 1u, abort_flag, a.err))) break;
                    if constexpr (BITS == 4) {
                        const int buffer = j % L::kBuffers * 2 + values;
                        if (lane == 0) asm volatile("st.shared.u32 [%0], %1;" ::"r"(base + L::kWide + 4 * buffer), "r"(values ? wide[1] : wide[0]) : "memory");
                        asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(base + L::kScales + buffer * (2 * kStep) + 8 * lane),
                                     "r"(values ? held[1][0] : held[0][0]), "r"(values ? held[1][1] : held[0][1])
                                     : "memory");
                        if (values == 0 && lane % 4 == 0)
                            info[j % kSlots * kSubs + lane / 4] =
                                PageData{__uint_as_float((wide[0] ? unit[0] - 11u : unit[0] + 9u) << 23),
                                         zero[1] ? kNegInf : (float)((int)unit[1] - (wide[1] ? 138 : 118)), now.live ? 1u : 2u};
                    } else if (values == 0 && lane < kSubs) {
                        const bool plain = now.live && now.ks == now.ks && now.vs == now.vs;
                        info[j % kSlots * kSubs + lane] = PageData{now.ks, plain ? log2f(now.vs) : 0.0f, plain ? 1u : now.live ? 0u : 2u};
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive_expect_tx(code_bar(kCFull, values, j), bytes);
                    __syncwarp();
                    if (copies) {
                        const uint8_t* from = BITS == 4 ? a.c.data + now.from + values * part : (values ? a.c.v : a.c.k) + now.from;
                        bulk_load(base + L::kCodes + (j % L::kBuffers * 2 + values) * L::kCodeBytes + lane * kTokens * (D * BITS / 8), from, part,
                                  code_bar(kCFull, values, j));
                    }
                    issued[values] = j + 1;
                }
                if (!ok) break;
                now = next;
            }
            // Copies in flight land before the CTA may leave.
            if (lane < 2)
                for (int j = max(0, issued[lane] - L::kBuffers); j < issued[lane]; ++j) drain(code_bar(kCFull, lane, j), code_parity(j), a.err);
        }
        __syncwarp();
    } else {
        more_registers<kSoftRegs>();
        if (which < tiles) {
        // ---------------- softmax: one row a thread ----------------
        const uint32_t quarter = (uint32_t)(warp % 4 * 32) << 16;
        const uint32_t s_at = tmem + which * kStep + quarter, o_at = tmem + 2 * kStep + which * kStep + quarter;
        const int first = tile.r0 + which * kTile, last = min(first + kTile, tile.nrows) - 1;
        const int full_lo = tile.row_lo(a, last), full_hi = tile.row_hi(a, first);
        const bool live = my_row < tile.nrows;
        const int lo = live ? tile.row_lo(a, my_row) : 0, hi = live ? tile.row_hi(a, my_row) : tile.hi;
        // The row's own largest score s_j and s_j + log2 of its page's value scale
        // v_j so far, of tokens that it sees: l sums exp2(s_j - m) in binary32, the
        // second product takes 2^15 exp2(s_j + log2 v_j - mv) as binary16.
        float m = kLowest, mv = kLowest, l = 0.0f;
        bool ok = true;
        for (int j = 0; j < blocks; ++j) {
            if (!(ok = warp_wait(bars + 8 * (kSFull + which), (uint32_t)j & 1u, abort_flag, a.err))) break;
            tc_fence_after();
            const PageData* page = info + j % kSlots * kSubs;
            const int tok = tok_begin + j * kStep;
            uint32_t v[4][32];   // the row's scores, all in registers
            tmem_ld_32x32b_x32(s_at, v[0]);
            tmem_ld_32x32b_x32(s_at + 32, v[1]);
            uint32_t plain = 1;
#pragma unroll
            for (int b = 0; b < kSubs; ++b) plain &= page[b].plain;
            // Factors stay above 0, so that -inf times one stays that; a NaN
            // scale's tokens are NaN or -inf already.
            auto factor = [&](int b) {
                const float f = row_scale * page[b].ks;
                return f >= 1.1754943508222875e-38f ? f : 1.1754943508222875e-38f;
            };
            const bool hidden = tok < full_lo || tok + kStep > full_hi;
            const int first_seen = lo - tok, end_seen = hi - tok;
            float top = kLowest, top_v = kLowest;
#pragma unroll
            for (int half = 0; half < 2; ++half) {   // the second half loads meanwhile
                tmem_ld_wait_for(v[2 * half]);
                tmem_ld_wait_for(v[2 * half + 1]);
                if (half == 0) {
                    tmem_ld_32x32b_x32(s_at + 64, v[2]);
                    tmem_ld_32x32b_x32(s_at + 96, v[3]);
                }
                if (hidden) {   // hidden tokens: -inf
#pragma unroll
                    for (int e = 64 * half; e < 64 * half + 64; ++e)
                        if (e < first_seen || e >= end_seen) v[e / 32][e % 32] = 0xFF800000u;
                    asm volatile("");
                }
                if (!(plain & 1u)) {   // pages that are not there: hidden; that read as NaN: NaN, where seen
#pragma unroll
                    for (int b = 4 * half; b < 4 * half + 4; ++b) {
                        const uint32_t kind = page[b].plain;
                        if (kind == 1u) continue;
#pragma unroll
                        for (int e = 0; e < kSub; ++e) {
                            uint32_t& x = v[b / 2][b % 2 * 16 + e];
                            if (kind == 2u) x = 0xFF800000u;
                            else if (x != 0xFF800000u) x = 0x7FC00000u;
                        }
                    }
                    asm volatile("");
                }
#pragma unroll
                for (int b = 4 * half; b < 4 * half + 4; ++b) {
                    const uint32_t* x = &v[b / 2][b % 2 * 16];
                    auto at = [&](int e) { return __uint_as_float(x[e]); };
                    const float t0 = max3(max3(at(0), at(1), at(2)), at(3), at(4)), t1 = max3(max3(at(5), at(6), at(7)), at(8), at(9));
                    const float t2 = max3(max3(at(10), at(11), at(12)), at(13), at(14));
                    const float t = max3(max3(t0, t1, t2), at(15), at(15)) * factor(b);
                    top = fmaxf(top, t);
                    top_v = fmaxf(top_v, t + page[b].log_v);
                }
            }
            // The sums so far are brought to new maxima only when one is passed (that of
            // the scores, which the binary32 sum is relative to, by more); of 4 bits in
            // the rows alone that passed one, whatever their neighbours do.
            const bool passed = top > m + 16.0f || top_v > mv + kLag;
            if (__any_sync(0xFFFFFFFFu, passed)) {
                const bool mine = BITS == 8 || passed;
                const float nm = mine ? fmaxf(m, top) : m, nmv = mine ? fmaxf(mv, top_v) : mv, keep = exp2_approx(mv - nmv);
                l *= exp2_approx(m - nm);
                m = nm;
                mv = nmv;
                if (j > 0) {
                    if (!(ok = warp_wait(bars + 8 * (kODone + which), (uint32_t)(j - 1) & 1u, abort_flag, a.err))) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D / 16; ++c) {
                        uint32_t y[16];
                        tmem_ld_x16(o_at + 16 * c, y);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * keep);
                        tmem_st_x16(o_at + 16 * c, y);
                    }
                }
            }
            // A page's value scale is taken for one at which a weight of 1 is 2^-60 of the
            // row's largest if it is less (0 too): none of its weights is a binary16
            // above 0, and their sum can be had from the same exponentials.
            const float shift_v = 15.0f - mv, least = 15.0f - 60.0f - m;
            float sum[2] = {0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t p[16];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const PageData& pd = page[2 * c + b];
                    const float f = factor(2 * c + b), shift = fmaxf(pd.log_v + shift_v, least);
                    const float2 f2 = make_float2(f, f), shift2 = make_float2(shift, shift);
                    float2 s2 = make_float2(0.0f, 0.0f), s3 = s2;
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        const uint32_t* x = &v[c][16 * b + e];
                        float2 w = __ffma2_rn(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])), f2, shift2);
                        float2 y = __ffma2_rn(make_float2(__uint_as_float(x[2]), __uint_as_float(x[3])), f2, shift2);
                        w = make_float2(exp2_approx(w.x), exp2_approx(w.y));
                        y = make_float2(exp2_approx(y.x), exp2_approx(y.y));
                        s2 = __fadd2_rn(s2, w);
                        s3 = __fadd2_rn(s3, y);
                        p[8 * b + e / 2] = pack2<__half>(w.x, w.y);
                        p[8 * b + e / 2 + 1] = pack2<__half>(y.x, y.y);
                    }
                    s2 = __fadd2_rn(s2, s3);
                    sum[b] = fmaf(s2.x + s2.y, exp2_approx(-shift - m), sum[b]);
                }
                tmem_st_x16(s_at + 16 * c, p);   // over scores that are in registers
                if (c & 1) {
                    tmem_st_wait();
                    tc_fence_before();
                    warp_arrive(bars + 8 * (kPFull + 2 * which + c / 2));
                }
            }
            l += sum[0] + sum[1];
        }
        if (ok && blocks > 0) ok = warp_wait(bars + 8 * (kODone + which), (uint32_t)(blocks - 1) & 1u, abort_flag, a.err);
        tc_fence_after();
        if (ok) {
            [[maybe_unused]] const int64_t o_bytes =
                ((a.b.rows - 1) * a.O.row + (a.q_heads - 1) * a.O.head + D) * (int64_t)sizeof(T);
            const bool whole = tile.active == 1;
            // O is in units of 2^(mv - 15), results and partial sums in those of 2^m, by
            // two factors that are both in range.
            const bool none = blocks == 0 || l == 0.0f;
            const float half_unit = exp2_approx(0.5f * (mv - m)), unit = half_unit * (whole ? 1.0f / kPScale / l : 1.0f / kPScale);
            T* dst = live ? out_row<T>(a, tile, h, my_row) : nullptr;
            float* part = whole ? nullptr : a.partial + (((int64_t)u * a.c.heads + h) * a.splits + split) * ((int64_t)kRows * (D + 2));
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t v[32] = {};
                if (blocks > 0) tmem_ld_32x32b_x32(o_at + 32 * c, v);
                tmem_ld_wait();
                float y[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) y[e] = none ? 0.0f : __uint_as_float(v[e]) * half_unit * unit;
                if (!live) {
                } else if (!whole) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        if (GEMM_DBG_OK(part + (int64_t)threadIdx.x * D + 32 * c + e, a.partial, a.partial_bytes, 16))
                            *reinterpret_cast<float4*>(part + (int64_t)threadIdx.x * D + 32 * c + e) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
                } else if (o_vec) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        if (GEMM_DBG_OK(dst + 32 * c + e, a.O.p, o_bytes, 16))
                            *reinterpret_cast<uint4*>(dst + 32 * c + e) =
                                make_uint4(pack2<T>(y[e], y[e + 1]), pack2<T>(y[e + 2], y[e + 3]), pack2<T>(y[e + 4], y[e + 5]), pack2<T>(y[e + 6], y[e + 7]));
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (GEMM_DBG_OK(dst + 32 * c + e, a.O.p, o_bytes, sizeof(T))) dst[32 * c + e] = from_float<T>(y[e]);
                }
                __syncwarp();
            }
            if (live && !whole && GEMM_DBG_OK(part + (int64_t)kRows * D + 2 * threadIdx.x, a.partial, a.partial_bytes, 8)) {
                part[(int64_t)kRows * D + 2 * threadIdx.x] = m;
                part[(int64_t)kRows * D + 2 * threadIdx.x + 1] = l;
            }
        }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kSoftWarps + kCacheWarps) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <typename T, int D, int BITS>
cudaError_t launch(const AttnArgs& a, const KvPlan& plan, cudaStream_t stream) {
    const bool o_vec = (reinterpret_cast<uintptr_t>(a.O.p) & 15u) == 0 && a.O.row % 8 == 0 && a.O.head % 8 == 0;
    kv_prompt_kernel<T, D, BITS><<<(unsigned)(plan.units * plan.splits * a.c.heads), kThreads, Smem<D, BITS>::kBytes, stream>>>(a, o_vec);
    return cudaGetLastError();
}

template <typename T, int D, int BITS>
cudaError_t allow_smem() {
    // The roles' shares of the registers would wait for ever if the launch had fewer.
    cudaFuncAttributes f;
    const cudaError_t e = cudaFuncGetAttributes(&f, kv_prompt_kernel<T, D, BITS>);
    if (e != cudaSuccess) return e;
    if (f.numRegs < kLaunchRegs) return cudaErrorInvalidConfiguration;
    return cudaFuncSetAttribute(kv_prompt_kernel<T, D, BITS>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D, BITS>::kBytes);
}

// Calls f with a kernel's type, head size and bits.
template <typename F>
cudaError_t with_kernel(ElemType type, int dim, int bits, F f) {
    using std::integral_constant;
    auto by_bits = [&](auto t, auto d) { return bits == 4 ? f(t, d, integral_constant<int, 4>()) : f(t, d, integral_constant<int, 8>()); };
    auto by_dim = [&](auto t) { return dim == 64 ? by_bits(t, integral_constant<int, 64>()) : by_bits(t, integral_constant<int, 128>()); };
    return type == ElemType::kBF16 ? by_dim(__nv_bfloat16()) : by_dim(__half());
}

}  // namespace

LIBGEMM_DEBUG_READER(kv_prompt_debug_flags)

cudaError_t kv_prompt_setup(int bits) {
    for (ElemType type : {ElemType::kBF16, ElemType::kF16})
        for (int dim : {64, 128}) {
            const cudaError_t e = with_kernel(type, dim, bits, [](auto t, auto d, auto b) {
                return allow_smem<decltype(t), decltype(d)::value, decltype(b)::value>();
            });
            if (e != cudaSuccess) return e;
        }
    return cudaSuccess;
}

cudaError_t launch_kv_prompt(const AttnArgs& a, ElemType type, const KvPlan& plan, cudaStream_t stream) {
    return with_kernel(type, a.c.dim, a.c.bits, [&](auto t, auto d, auto b) {
        return launch<decltype(t), decltype(d)::value, decltype(b)::value>(a, plan, stream);
    });
}

}  // namespace libgemm
