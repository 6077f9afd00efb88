// kv_prompt.cu -- attention of many query rows (prompts) over the paged 8-bit
// cache, on the 5th-generation tensor cores.
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
// Every wait is bounded; a role that gives up raises the abort flag, all stop,
// and the matrix unit is drained before tensor memory is freed.
#include "kv_attention.cuh"

namespace libgemm {
namespace {

constexpr int kTile = 128, kRows = 2 * kTile, kStep = 128;   // rows of a tile and a CTA, tokens of a block
constexpr int kSub = 16, kSubs = kStep / kSub;               // tokens that share a page for certain
constexpr int kSlots = 4;                                    // blocks whose page data are kept
constexpr int kSoftWarps = 8, kCacheWarps = 4, kThreads = (kSoftWarps + kCacheWarps + 4) * 32;
// Registers of a thread: launched with 128, then shared out among the roles
// (whole warpgroups), whose sum is that of the launch.
constexpr int kLaunchRegs = 128, kSoftRegs = 184, kCacheRegs = 104, kIssueRegs = 40;
static_assert(kSoftRegs * kSoftWarps + kCacheRegs * kCacheWarps + kIssueRegs * 4 <= kLaunchRegs * kThreads / 32, "");
constexpr int kSlab = kTile * 128;                           // 128 rows of 64 binary16

// What a softmax thread needs of 16 tokens: the key scale, log2 of the
// value scale (-inf for one of 0).
struct alignas(16) PageData {
    float ks, log_v;
    uint32_t plain;      // 1: there, and reads as numbers; 0: reads as NaN; 2: not there
};

template <int D>
struct Smem {
    static constexpr int kOperand = D / 64 * kSlab;          // 128 x D binary16
    static constexpr int kQ = 0, kK = 2 * kOperand, kV = kK + 2 * kOperand;
    static constexpr int kCodes = kV + 2 * kOperand, kInfo = kCodes + 2 * kStep * D;   // codes: keys, values
    static constexpr int kBars = kInfo + kSlots * kSubs * (int)sizeof(PageData);
    static constexpr int kBytes = kBars + 256 + 1024;        // and the alignment
};
// Barriers: keys and values full / empty (two buffers), per tile scores full,
// weights full (of the first and of the last 64 tokens), output done; codes
// full / empty (keys, values); the drain.
enum { kKFull = 0, kKEmpty = 2, kVFull = 4, kVEmpty = 6, kSFull = 8, kPFull = 10, kODone = 14, kCFull = 16, kCEmpty = 18, kDrain = 20 };

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

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1) kv_prompt_kernel(const AttnArgs a, bool o_vec) {
    using L = Smem<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    PageData* info = reinterpret_cast<PageData*>(smem + L::kInfo);
    const uint32_t bars = base + L::kBars;
    volatile int* abort_flag = &s_abort;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
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
            st_shared_v4(q0 + c / 8 * kSlab + swizzled(in_tile, c % 8), pack2<__half>(x.at(0) * down, x.at(1) * down),
                         pack2<__half>(x.at(2) * down, x.at(3) * down), pack2<__half>(x.at(4) * down, x.at(5) * down),
                         pack2<__half>(x.at(6) * down, x.at(7) * down));
        }
        fence_proxy_async_shared();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;

    if (warp >= kSoftWarps && warp < kSoftWarps + kCacheWarps) {
        // ---------------- the cache ----------------
        fewer_registers<kCacheRegs>();
        constexpr int kLanes = D / 16;                  // lanes of a token, 16 codes each
        constexpr int kPassRows = kCacheWarps * 32 / kLanes, kPasses = kStep / kPassRows;
        const int ct = threadIdx.x - kSoftWarps * 32;
        // A quarter of a warp holds halves of two neighbouring rows: its 16-byte
        // stores then meet all eight chunk positions of the swizzle.
        const int piece = D == 128 ? ct % 4 + 4 * (ct / 8 % 2) : ct % 4;
        const int sub_row = D == 128 ? ct / 16 * 2 + ct / 4 % 2 : ct / 4;
        uint4 w[kPasses];
        auto get = [&](int values, uint32_t parity) {
            if (!warp_wait(bars + 8 * (kCFull + values), parity, abort_flag, a.err)) return false;
            const uint32_t from = base + L::kCodes + values * (kStep * D) + sub_row * D + 16 * piece;
#pragma unroll
            for (int i = 0; i < kPasses; ++i) w[i] = lds128(from + i * kPassRows * D);
            return true;
        };
        auto put = [&](uint32_t to) {
            const int c = 2 * piece % 8;
            const uint32_t at = to + 2 * piece / 8 * kSlab + sub_row * 128, r = sub_row & 7;
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const uint32_t row = at + i * kPassRows * 128;
                st_shared_v4(row + ((c ^ r) << 4), codes01(w[i].x), codes23(w[i].x), codes01(w[i].y), codes23(w[i].y));
                st_shared_v4(row + (((c + 1) ^ r) << 4), codes01(w[i].z), codes23(w[i].z), codes01(w[i].w), codes23(w[i].w));
            }
            fence_proxy_async_shared();
        };
        for (int j = 0; j < blocks; ++j) {
            const int buf = j & 1;
            const uint32_t parity = (uint32_t)(j >> 1) & 1u;
            if (!get(0, (uint32_t)j & 1u)) break;
            warp_arrive(bars + 8 * kCEmpty);
            if (!warp_wait(bars + 8 * (kKEmpty + buf), parity ^ 1u, abort_flag, a.err)) break;
            put(base + L::kK + buf * L::kOperand);
            warp_arrive(bars + 8 * (kKFull + buf));
            if (!get(1, (uint32_t)j & 1u)) break;
            warp_arrive(bars + 8 * (kCEmpty + 1));
            if (!warp_wait(bars + 8 * (kVEmpty + buf), parity ^ 1u, abort_flag, a.err)) break;
            put(base + L::kV + buf * L::kOperand);
            warp_arrive(bars + 8 * (kVFull + buf));
        }
    } else if (warp >= kSoftWarps + kCacheWarps) {
        // ---------------- the matrix unit ----------------
        fewer_registers<kIssueRegs>();
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
            // ---------------- the copies: lane i < 8 looks after 16 tokens of a block ----------------
            [[maybe_unused]] const int64_t code_bytes = a.c.pages * a.c.heads * ((int64_t)D << log2);
            const int chunk = min(kStep, 1 << log2);   // tokens of one copy
            struct Sub { int64_t from; float ks, vs; bool live; };
            auto look = [&](int j) {
                Sub s{0, 0.0f, 0.0f, false};
                const int tok = tok_begin + j * kStep + lane * kSub;
                if (lane < kSubs && j < blocks && tile.page_seen(tok, log2)) {
                    const int64_t page = __ldg(table + (tok >> log2));
                    s.live = page >= 0 && page < a.c.pages;
                    if (!s.live) atomicOr(a.err, kErrIndex);
                    else {
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
                // the first 16 tokens of a page's part fetch all of it
                bool copies = now.live && lane * kSub % chunk == 0;
                if (copies) copies = GEMM_DBG_OK(a.c.k + now.from, a.c.k, code_bytes, chunk * D) && GEMM_DBG_OK(a.c.v + now.from, a.c.v, code_bytes, chunk * D);
                const uint32_t bytes = (uint32_t)(__popc(__ballot_sync(0xFFFFFFFFu, copies)) * chunk * D);
                bool ok = true;
#pragma unroll
                for (int values = 0; values < 2; ++values) {
                    // Page data of block j go where those of block j - 4 were: its keys' turn
                    // comes when the keys of j - 1 are taken, so the values of j - 4 are used up.
                    if (!(ok = warp_wait(bars + 8 * (kCEmpty + values), ((uint32_t)j & 1u) ^ 1u, abort_flag, a.err))) break;
                    if (values == 0 && lane < kSubs) {
                        const bool plain = now.live && now.ks == now.ks && now.vs == now.vs;
                        info[j % kSlots * kSubs + lane] = PageData{now.ks, plain ? log2f(now.vs) : 0.0f, plain ? 1u : now.live ? 0u : 2u};
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive_expect_tx(bars + 8 * (kCFull + values), bytes);
                    __syncwarp();
                    if (copies)
                        bulk_load(base + L::kCodes + values * (kStep * D) + lane * kSub * D, (values ? a.c.v : a.c.k) + now.from, chunk * D, bars + 8 * (kCFull + values));
                    issued[values] = j + 1;
                }
                if (!ok) break;
                now = next;
            }
            // Copies in flight land before the CTA may leave.
            if (lane < 2 && issued[lane] > 0) {
                drain(bars + 8 * (kCFull + lane), (uint32_t)(issued[lane] - 1) & 1u, a.err);
            }
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
            // the scores, which the binary32 sum is relative to, by more).
            if (__any_sync(0xFFFFFFFFu, top > m + 16.0f || top_v > mv + kLag)) {
                const float nm = fmaxf(m, top), nmv = fmaxf(mv, top_v), keep = exp2_approx(mv - nmv);
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

template <typename T, int D>
cudaError_t launch(const AttnArgs& a, const KvPlan& plan, cudaStream_t stream) {
    const bool o_vec = (reinterpret_cast<uintptr_t>(a.O.p) & 15u) == 0 && a.O.row % 8 == 0 && a.O.head % 8 == 0;
    kv_prompt_kernel<T, D><<<(unsigned)(plan.units * plan.splits * a.c.heads), kThreads, Smem<D>::kBytes, stream>>>(a, o_vec);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t allow_smem() {
    // The roles' shares of the registers would wait for ever if the launch had fewer.
    cudaFuncAttributes f;
    const cudaError_t e = cudaFuncGetAttributes(&f, kv_prompt_kernel<T, D>);
    if (e != cudaSuccess) return e;
    if (f.numRegs < kLaunchRegs) return cudaErrorInvalidConfiguration;
    return cudaFuncSetAttribute(kv_prompt_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kBytes);
}

}  // namespace

LIBGEMM_DEBUG_READER(kv_prompt_debug_flags)

cudaError_t kv_prompt_setup() {
    cudaError_t e = allow_smem<__nv_bfloat16, 64>();
    if (e == cudaSuccess) e = allow_smem<__nv_bfloat16, 128>();
    if (e == cudaSuccess) e = allow_smem<__half, 64>();
    if (e == cudaSuccess) e = allow_smem<__half, 128>();
    return e;
}

cudaError_t launch_kv_prompt(const AttnArgs& a, ElemType type, const KvPlan& plan, cudaStream_t stream) {
    if (type == ElemType::kBF16)
        return a.c.dim == 128 ? launch<__nv_bfloat16, 128>(a, plan, stream) : launch<__nv_bfloat16, 64>(a, plan, stream);
    return a.c.dim == 128 ? launch<__half, 128>(a, plan, stream) : launch<__half, 64>(a, plan, stream);
}

}  // namespace libgemm
