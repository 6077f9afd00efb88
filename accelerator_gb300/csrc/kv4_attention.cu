// kv4_attention.cu -- attention of few query rows over the paged 4-bit cache.
//
// For each query row  o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale * q.k_j
// - m), in one pass over the tokens with the running maximum m and sum, as over
// the 8-bit cache (kv_attention.cu), whose tiles, splits and joining it has.
// What differs is what 4 bits allow.
//
// A code u = c + 8 is a nibble, and a word that is masked with 0x000F000F or
// 0x00F000F0 holds two of them as binary16 numbers below the normal range, u *
// 2^-24 or u * 2^-20, which the matrix instruction multiplies exactly: a word of
// eight codes takes five instructions (one shift, four masks), and none of them
// converts.  The powers of two go onto the queries (16 times as large where the
// codes are 2^-24) and the results.  The 8 in u goes out of the sums: of the
// scores by where they begin, at -8 times the sum of the query, and of the results
// by a product more, whose 16 rows are ones: it sums the weights as they were
// rounded, so that their rounding errors meet c and not u.
//
// Every token has its own scales.  A page and head's codes and scales lie in one
// piece, and one bulk copy brings them.
#include "kv_attention.cuh"

namespace libgemm {
namespace {

constexpr int kWarps = 4;        // warps that compute; one more copies
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kSub = 16;         // tokens of one product, all of one page
constexpr int kSubs = 2;         // a warp takes this many times 16 tokens at once
constexpr int kStep = kWarps * kSubs * kSub;   // tokens of a stage
constexpr int resident(int nq) { return nq == 1 ? 3 : 2; }   // CTAs of an SM
constexpr int ring_bytes(int nq) { return nq == 1 ? 70 * 1024 : 102 * 1024; }
// Weights enter the second product relative to 2^12 for the row's largest: 2^3.9
// over it still fit binary16, so that a row's sums are seldom brought to a new
// maximum, and 2^-26 under it is still a normal number.
constexpr float kTopP = 4096.0f;
// A row's largest weight times value scale counts as this if it is less: the
// factor up to kTopP stays finite when a weight of up to kMostP multiplies it.
constexpr float kLeastP = 3.1554436e-30f;   // 2^-98
constexpr int kMaxCluster = 8;

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}
// A bfloat16 in shared memory.
__device__ __forceinline__ float lds_bf16(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
    return __uint_as_float((uint32_t)v << 16);
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
// D / 8 bytes.
template <int D>
__device__ __forceinline__ void load_words(uint32_t addr, uint32_t (&w)[D / 32]) {
    if constexpr (D == 128) {
        const uint4 v = lds128(addr);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
        const uint2 v = lds64(addr);
        w[0] = v.x, w[1] = v.y;
    }
}
constexpr uint32_t kLow = 0x000F000Fu, kHigh = 0x00F000F0u;   // u * 2^-24, u * 2^-20

template <int D, int NQ>
struct Ring {
    static constexpr int kStageBytes = kStep * (D + 4);
    static constexpr int kStages = ring_bytes(NQ) / kStageBytes;   // 4 or 6 for 128, 8 or 12 for 64
    // [stages][pages' records], then a word a stage, then the barriers
    static constexpr int kLiveAt = kStages * kStageBytes;
    static constexpr int kBarsAt = kLiveAt + (4 * kStages + 15) / 16 * 16;
    static constexpr int kAbortAt = kBarsAt + 16 * kStages;
    static constexpr int kBytes = kAbortAt + 16;
};

// The 8 x 8 binary16 matrix that a warp holds in fragments (lane 4 g + t has
// row g, columns 2t and 2t + 1), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// A tile of 8 * NQ rows over a share of its tokens.  One warp copies pages into a
// ring of stages of 128 tokens, four take 32 tokens of each stage; the tokens' side
// is the 16-row operand of both products and the queries its eight columns: S^T =
// K Q^T, then O^T = V^T P^T, for which the weights are turned over in registers.
template <typename T, int D, int NQ>
__global__ void __launch_bounds__(kThreads, resident(NQ)) kv4_attention_kernel(const AttnArgs a) {
    using R = Ring<D, NQ>;
    constexpr int kRows = 8 * NQ, kLd = D + 4, kWords = D / 32;
    static_assert(kWarps * kRows * (kLd + 2) * 4 + 8 * kRows <= R::kLiveAt, "the joining reuses the ring");
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t ring = smem_u32(smem), bars = ring + R::kBarsAt;   // full[stages], empty[stages]
    uint32_t* live_subs = reinterpret_cast<uint32_t*>(smem + R::kLiveAt);   // which 16s of a stage are there
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + R::kAbortAt);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int u = blockIdx.x / a.splits, split = blockIdx.x % a.splits, h = blockIdx.y;
    const bool cluster = a.splits > 1 && !a.partial;
    Tile tile;
    // A cluster's CTAs have one tile: they leave here together or not at all.
    if (!tile.find(a, u, kRows, kStep, h == 0 && split == 0) || (!cluster && split >= tile.active)) return;
    grid_launch_dependents();   // a joining launch may start its set-up
    const int step_begin = min(tile.steps, split * tile.per);
    const int steps = min(tile.steps, step_begin + tile.per) - step_begin;
    const int tok_begin = tile.tok0 + step_begin * kStep;
    const int log2 = a.c.page_log2, page_tokens = 1 << log2, record = (D + 4) << log2;
    if (threadIdx.x == 0) {
        for (int s = 0; s < R::kStages; ++s) {
            mbar_init(bars + 8 * s, 1);
            mbar_init(bars + 8 * (R::kStages + s), kWarps);
        }
        *abort_flag = 0;
        mbar_fence_init();
    }
    __syncthreads();

    float* s_o = reinterpret_cast<float*>(smem);                     // [warps][rows][kLd]
    float* s_m = s_o + kWarps * kRows * kLd;                      // [warps][rows]
    float* s_l = s_m + kWarps * kRows;
    if (warp == kWarps) {
        // ---- copies: lane i looks up 16 tokens, those of four stages at a time ----
        static_assert(kWarps * kSubs == 8, "");
        const int32_t* table = a.b.table + tile.seq * a.b.width;
        [[maybe_unused]] const int64_t extent = a.c.pages * a.c.heads * a.c.record();
        bool live = false;
        const uint8_t* from = nullptr;
        uint32_t phase = 0;
        int stage = 0, issued = 0;
        for (int s = 0; s < steps; ++s) {
            if (s % 4 == 0) {
                const int tok = tok_begin + s * kStep + lane * kSub;
                live = tile.page_seen(tok, log2);
                const int64_t page = live ? __ldg(table + (tok >> log2)) : 0;
                if (live && (page < 0 || page >= a.c.pages)) {
                    atomicOr(a.err, kErrIndex);
                    live = false;
                }
                from = a.c.data + (page * a.c.heads + h) * record;
            }
            if (!warp_wait(bars + 8 * (R::kStages + stage), phase ^ 1u, abort_flag, a.err)) break;
            const int sub = lane - s % 4 * 8;   // this lane's part of the stage, if it has one
            const bool here = sub >= 0 && sub < 8 && live;
            bool copies = here && sub * kSub % page_tokens == 0;   // a page's first 16 tokens fetch all of it
            if (copies) copies = GEMM_DBG_OK(from, a.c.data, extent, record);
            const unsigned there = __ballot_sync(0xFFFFFFFFu, here), parts = __popc(__ballot_sync(0xFFFFFFFFu, copies));
            if (copies) bulk_load(ring + stage * R::kStageBytes + (sub * kSub >> log2) * record, from, record, bars + 8 * stage);
            __syncwarp();
            if (lane == 0) {
                live_subs[stage] = there >> (s % 4 * 8);
                mbar_arrive_expect_tx(bars + 8 * stage, parts * record);
            }
            ++issued;
            if (++stage == R::kStages) stage = 0, phase ^= 1u;
        }
        // Copies in flight land before the CTA may leave or reuse the ring.
        if (lane == 0)
            for (int s = max(0, issued - R::kStages); s < issued; ++s) drain(bars + 8 * (s % R::kStages), (uint32_t)(s / R::kStages) & 1u, a.err);
        __syncwarp();
        __syncthreads();   // the ring is free
        __syncthreads();   // the warps' results are in it
    } else {
        // Query row 8n + g as the column g of B.  A lane's part of a row is 8
        // neighbours of each 32: elements e and e + 4 a word's two halves hold
        // together.  Rows are brought to [2^11, 2^12) by a power of two, so that 16
        // times that is binary16 (exact, but for elements under 2^-25 of the row's
        // largest, whose error stays under 2^-36 of it).
        uint32_t qf[NQ][2 * kWords][2];
        float factor[NQ][2], begin[NQ][4];      // of the rows 8n + 2t, + 1, whose scores a lane gets
        int row_lo[NQ][2], row_hi[NQ][2];
        [[maybe_unused]] const int64_t q_bytes =
            ((a.b.rows - 1) * a.Q.row + (a.q_heads - 1) * a.Q.head + D) * (int64_t)sizeof(T);
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const unsigned r = tile.r0 + 8 * n + g;
            const bool live = r < (unsigned)tile.nrows;
            const T* p = static_cast<const T*>(a.Q.p) + (int64_t)(tile.row0 + (live ? r / a.share : 0)) * a.Q.row +
                         (int64_t)(h * a.share + (live ? r % a.share : 0)) * a.Q.head;
            Eight<T> x[kWords] = {};
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                const T* pe = p + 32 * i + 8 * t;
                if (live && GEMM_DBG_OK(pe, a.Q.p, q_bytes, 16)) x[i] = load_eight(pe, a.q_vec);
#pragma unroll
                for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[i].at(e)));
            }
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            // its biased exponent, in the range in which both powers below are normal
            const int k = top < INFINITY ? max(12, min(249, (int)(__float_as_uint(top) >> 23))) : 127;
            const float down = __uint_as_float((uint32_t)(265 - k) << 23) * (a.scale_log2 < 0.0f ? -1.0f : 1.0f);   // 2^(11 + 127 - k)
            const float up = __uint_as_float((uint32_t)(k + 5) << 23);   // 2^(k - 127 - 11 + 20 - 4): the codes' 2^-20, 2^4 of it with the key's scale
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kWords; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float by = e & 1 ? down : 16.0f * down, a0 = x[i].at(e) * by, a1 = x[i].at(e + 4) * by;
                    const uint32_t two = pack2<__half>(a0, a1);
                    const float2 held = __half22float2(*reinterpret_cast<const __half2*>(&two));
                    qf[n][2 * i + e / 2][e & 1] = two;
                    sum += (held.x + held.y) * (e & 1 ? 1.0f : 0.0625f);
                }
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                begin[n][i] = begin[n][2 + i] = -8.0f * 9.5367431640625e-7f * __shfl_sync(0xFFFFFFFFu, sum, 4 * (2 * t + i));   // 2^-20
                // above 0, so that a hidden token's -inf stays that
                factor[n][i] = fmaxf(fabsf(a.scale_log2) * __shfl_sync(0xFFFFFFFFu, up, 4 * (2 * t + i)), 1.1754943508222875e-38f);
                // rows past the last one see all: they are not stored
                const int rr = tile.r0 + 8 * n + 2 * t + i;
                row_lo[n][i] = rr < tile.nrows ? tile.row_lo(a, rr) : 0;
                row_hi[n][i] = rr < tile.nrows ? tile.row_hi(a, rr) : tile.hi;
            }
        }
        // tokens that every row of the tile sees
        const int full_lo = tile.row_lo(a, min(tile.r0 + kRows, tile.nrows) - 1);
        const int full_hi = tile.row_hi(a, tile.r0);

        constexpr int MT = D / 16;      // row tiles of O^T: row g of tile 2i + x is d = 64 (i / 2) + 8g + 4 (i % 2) + 2x, row g + 8 the next
        // A row's sums: l of the weights exp2(s_j - m) in binary32, o of those times
        // their token's value scale v_j times up = 2^12 / r as binary16, and ones of these
        // alone, where m and r are the row's own largest s_j and exp2(s_j - m) * v_j so
        // far, of tokens that it sees (r at least kLeastP).
        float o[NQ][MT][4], ones[NQ][4], m[NQ][2], l[NQ][2], up[NQ][2];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
#pragma unroll
            for (int i = 0; i < MT; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.0f;
            ones[n][0] = ones[n][1] = ones[n][2] = ones[n][3] = 0.0f;
            m[n][0] = m[n][1] = kLowest;
            l[n][0] = l[n][1] = 0.0f;
            up[n][0] = up[n][1] = kTopP / kLeastP;
        }

        uint32_t phase = 0;
        int stage = 0;
        for (int s = 0; s < steps; ++s) {
            if (!warp_wait(bars + 8 * stage, phase, abort_flag, a.err)) break;
            const int tok = tok_begin + s * kStep + warp * (kSubs * kSub);
            if (tok < tile.hi) {
                const uint32_t subs = live_subs[stage] >> (warp * kSubs);
                uint32_t base[kSubs];   // of each 16's page, and what of it comes before them
                int in[kSubs];
#pragma unroll
                for (int b = 0; b < kSubs; ++b) {
                    const int at = warp * (kSubs * kSub) + b * kSub;
                    base[b] = ring + stage * R::kStageBytes + (at >> log2) * record;
                    in[b] = at & (page_tokens - 1);
                }
                // scores of tokens 16b + g and 16b + g + 8 for the rows 2t, 2t + 1
                float sc[kSubs][NQ][4], vs[kSubs][2], held[kSubs][2], nan_sum = 0.0f;
#pragma unroll
                for (int b = 0; b < kSubs; ++b) {
                    const uint32_t kat = base[b] + in[b] * (D / 2) + g * (D / 2) + t * (D / 8);
                    const uint32_t sat = base[b] + page_tokens * D + 2 * (in[b] + g);
                    uint32_t w0[kWords], w1[kWords];
                    load_words<D>(kat, w0);
                    load_words<D>(kat + 8 * (D / 2), w1);
                    const float ks[2] = {lds_bf16(sat) * 16.0f, lds_bf16(sat + 16) * 16.0f};
                    vs[b][0] = lds_bf16(sat + 2 * page_tokens), vs[b][1] = lds_bf16(sat + 2 * page_tokens + 16);
                    nan_sum += fabsf(vs[b][0]) + fabsf(vs[b][1]);
                    // finite, whatever a token has that no row sees, so that a weight of 0 stays 0
                    held[b][0] = fminf(fabsf(vs[b][0]), 3.3895314e38f), held[b][1] = fminf(fabsf(vs[b][1]), 3.3895314e38f);
                    float part[NQ][2][4];
                    constexpr float kZero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int i = 0; i < kWords; ++i)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const uint32_t lo = w0[i] >> (8 * x), hi = w1[i] >> (8 * x);
#pragma unroll
                            for (int n = 0; n < NQ; ++n)
                                mma_16816_from(part[n][x], i > 0 ? part[n][x] : x ? kZero : begin[n], lo & kLow, hi & kLow, lo & kHigh, hi & kHigh,
                                               qf[n][2 * i + x][0], qf[n][2 * i + x][1]);
                        }
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sc[b][n][e] = (part[n][0][e] + part[n][1][e]) * ks[e >> 1];
                }
                // Tokens that some row does not see, pages that do not exist.
                if (tok < full_lo || tok + kSubs * kSub > full_hi || (subs & 3u) != 3u) {
#pragma unroll
                    for (int b = 0; b < kSubs; ++b)
#pragma unroll
                        for (int n = 0; n < NQ; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int j = tok + 16 * b + g + 8 * (e >> 1);
                                if (j < row_lo[n][e & 1] || j >= row_hi[n][e & 1] || !(subs >> b & 1u)) sc[b][n][e] = kNegInf;
                            }
                    asm volatile("");   // a branch: few tokens come here
                }
                // A weight, and it with its token's value scale, relative to the row's largest.
                float w[kSubs][NQ][4], p[kSubs][NQ][4];
                auto weigh = [&] {   // returns the largest weight of either product
                    float most = 0.0f;
#pragma unroll
                    for (int b = 0; b < kSubs; ++b)
#pragma unroll
                        for (int n = 0; n < NQ; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                w[b][n][e] = exp2_approx(fmaf(sc[b][n][e], factor[n][e & 1], -m[n][e & 1]));
                                p[b][n][e] = w[b][n][e] * up[n][e & 1] * held[b][e >> 1];   // (0 of a weight of 0)
                                most = max3(most, w[b][n][e], p[b][n][e]);
                            }
                    return most;
                };
                // A row's sums so far are brought to a new maximum only when it is passed
                // by so much that a weight might not fit binary16, whatever the other
                // rows do: a row's result does not depend on its neighbours.
                const bool nan = nan_sum != nan_sum;
                if (__any_sync(0xFFFFFFFFu, weigh() > kMostP || nan)) {
#pragma unroll
                    for (int n = 0; n < NQ; ++n) {
                        float grow[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            auto across = [](float x) {   // the largest of the lanes that have this row
                                x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
                                x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
                                return fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
                            };
                            float most = 0.0f;
#pragma unroll
                            for (int b = 0; b < kSubs; ++b) most = max3(max3(most, w[b][n][i], p[b][n][i]), w[b][n][2 + i], p[b][n][2 + i]);
                            const bool passed = across(most) > kMostP;
                            // (every lane takes part in every exchange, also those whose row stays)
                            const float highest = across(fmaxf(fmaxf(sc[0][n][i], sc[0][n][2 + i]), fmaxf(sc[1][n][i], sc[1][n][2 + i])) * factor[n][i]);
                            const float top = passed ? fmaxf(highest, m[n][i]) : m[n][i];
                            const float keep = exp2_approx(m[n][i] - top), sums = keep * __fdividef(kTopP, up[n][i]);
                            m[n][i] = top;
                            l[n][i] *= keep;
                            float rel = 0.0f;
#pragma unroll
                            for (int b = 0; b < kSubs; ++b)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    if (sc[b][n][2 * e + i] != kNegInf) rel = fmaxf(rel, exp2_approx(fmaf(sc[b][n][2 * e + i], factor[n][i], -top)) * held[b][e]);
                            rel = across(rel);
                            rel = max3(rel, sums, kLeastP);
                            if (passed) up[n][i] = __fdividef(kTopP, rel);
                            grow[i] = passed ? __fdividef(sums, rel) : 1.0f;   // 1 at most
                        }
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            o[n][i][0] *= grow[0], o[n][i][1] *= grow[1];
                            o[n][i][2] *= grow[0], o[n][i][3] *= grow[1];
                        }
                        ones[n][0] *= grow[0], ones[n][1] *= grow[1];
                    }
                    weigh();
                    // values that read as NaN: for the rows that see them alone
#pragma unroll
                    for (int b = 0; b < kSubs; ++b)
#pragma unroll
                        for (int n = 0; n < NQ; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (vs[b][e >> 1] != vs[b][e >> 1]) p[b][n][e] = sc[b][n][e] == kNegInf ? 0.0f : vs[b][e >> 1];
                }
#pragma unroll
                for (int b = 0; b < kSubs; ++b) {
                    const uint32_t vat = base[b] + (page_tokens + in[b]) * (D / 2) + lane * (D / 8);
                    uint32_t w0[kWords], w1[kWords];   // tokens 2t, 2t + 1; those 8 on
                    load_words<D>(vat, w0);
                    load_words<D>(vat + 4 * D, w1);
                    // Binary16 under 2^16, normal down to 2^-26 of the row's largest.
                    uint32_t pt[NQ][2];
#pragma unroll
                    for (int n = 0; n < NQ; ++n) {
                        l[n][0] += w[b][n][0] + w[b][n][2];
                        l[n][1] += w[b][n][1] + w[b][n][3];
                        pt[n][0] = transpose8(pack2<__half>(p[b][n][0], p[b][n][1]));
                        pt[n][1] = transpose8(pack2<__half>(p[b][n][2], p[b][n][3]));
                        constexpr uint32_t kOne = 0x3C003C00u;
                        mma_16816<__half>(ones[n], kOne, kOne, kOne, kOne, pt[n][0], pt[n][1]);
                    }
#pragma unroll
                    for (int i = 0; i < kWords; ++i)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const uint32_t lo = w0[i] >> (8 * x), hi = w1[i] >> (8 * x);
#pragma unroll
                            for (int n = 0; n < NQ; ++n)
                                mma_16816<__half>(o[n][2 * i + x], lo & kLow, lo & kHigh, hi & kLow, hi & kHigh, pt[n][0], pt[n][1]);
                        }
                }
            }
            warp_arrive(bars + 8 * (R::kStages + stage));
            if (++stage == R::kStages) stage = 0, phase ^= 1u;
        }
        __syncthreads();   // the ring is free: every copy has landed and been used

        // Join the warps: each has a maximum, a sum and unnormalised outputs.
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int at = warp * kRows + 8 * n + 2 * t + i;
                const float unit = 1.0f / up[n][i], eight = 8.0f * ones[n][i];
                l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], 4);
                l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], 8);
                l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], 16);
                if (g == 0) s_m[at] = m[n][i], s_l[at] = l[n][i];
#pragma unroll
                for (int e = 0; e < kWords; ++e) {
                    // 2^24 and 2^20, less the codes' 8
                    auto value = [&](int x, int row) { return fmaf(o[n][2 * e + x][2 * row + i], row ? 1048576.0f : 16777216.0f, -eight) * unit; };
                    *reinterpret_cast<float4*>(s_o + at * kLd + 64 * (e / 2) + 8 * g + 4 * (e % 2)) =
                        make_float4(value(0, 0), value(0, 1), value(1, 0), value(1, 1));
                }
            }
        __syncthreads();
    }

    [[maybe_unused]] const int64_t o_bytes =
        ((a.b.rows - 1) * a.O.row + (a.q_heads - 1) * a.O.head + D) * (int64_t)sizeof(T);
    const int rows = min(tile.nrows - tile.r0, kRows);
    const bool whole = a.splits == 1 || (!cluster && tile.active == 1);
    float* part = a.partial ? a.partial + (((int64_t)u * a.c.heads + h) * a.splits + split) * (kRows * (D + 2)) : nullptr;
    for (int i = threadIdx.x; i < rows * D; i += kThreads) {
        const int r = i / D, d = i % D;
        float top = s_m[r];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_m[w * kRows + r]);
        float sum = 0.0f, acc = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = exp2_approx(s_m[w * kRows + r] - top);
            sum = fmaf(f, s_l[w * kRows + r], sum);
            acc = fmaf(f, s_o[(w * kRows + r) * kLd + d], acc);
        }
        if (whole) {
            T* dst = out_row<T>(a, tile, h, tile.r0 + r) + d;
            if (GEMM_DBG_OK(dst, a.O.p, o_bytes, sizeof(T))) *dst = from_float<T>(sum == 0.0f ? 0.0f : acc / sum);
        } else if (cluster) {
            s_o[r * kLd + d] = acc;   // warp 0's place: read by this thread alone so far
            if (d == 0) {
                float* ml = s_l + kWarps * kRows + 2 * r;
                ml[0] = top, ml[1] = sum;
            }
        } else {
            if (GEMM_DBG_OK(part + i, a.partial, a.partial_bytes, 4)) part[i] = acc;
            if (d == 0 && GEMM_DBG_OK(part + kRows * D + 2 * r, a.partial, a.partial_bytes, 8))
                part[kRows * D + 2 * r] = top, part[kRows * D + 2 * r + 1] = sum;
        }
    }
    if (!cluster) return;
    // The cluster's CTAs each join a share of the results, in split order.
    cluster_sync();
    const int share = (rows * D + a.splits - 1) / a.splits;
    for (int i = split * share + threadIdx.x; i < min(rows * D, (split + 1) * share); i += kThreads) {
        const int r = i / D, d = i % D;
        const uint32_t ml = smem_u32(s_l + kWarps * kRows + 2 * r), at = smem_u32(s_o + r * kLd + d);
        float tops[kMaxCluster], sums[kMaxCluster], accs[kMaxCluster], top = kLowest;
#pragma unroll
        for (int s = 0; s < kMaxCluster; ++s) {
            if (s >= tile.active) break;
            tops[s] = ld_cluster_f32(mapa_shared(ml, s));
            sums[s] = ld_cluster_f32(mapa_shared(ml + 4, s));
            accs[s] = ld_cluster_f32(mapa_shared(at, s));
            top = fmaxf(top, tops[s]);
        }
        float sum = 0.0f, acc = 0.0f;
#pragma unroll
        for (int s = 0; s < kMaxCluster; ++s) {
            if (s >= tile.active) break;
            const float f = exp2_approx(tops[s] - top);
            sum = fmaf(f, sums[s], sum);
            acc = fmaf(f, accs[s], acc);
        }
        T* dst = out_row<T>(a, tile, h, tile.r0 + r) + d;
        if (GEMM_DBG_OK(dst, a.O.p, o_bytes, sizeof(T))) *dst = from_float<T>(sum == 0.0f ? 0.0f : acc / sum);
    }
    cluster_sync();   // no CTA leaves while another reads its results
}

template <typename T, int D, int NQ>
cudaError_t launch(const AttnArgs& a, const KvPlan& plan, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(plan.units * plan.splits), (unsigned)a.c.heads);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Ring<D, NQ>::kBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = a.partial ? 1 : (unsigned)plan.splits;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv4_attention_kernel<T, D, NQ>, a);
}

// Calls f with a kernel's type, head size and eights of rows.
template <typename F>
cudaError_t with_kernel(ElemType type, int dim, int rows, F f) {
    auto by_rows = [&](auto t, auto d) {
        return rows == 8 ? f(t, d, std::integral_constant<int, 1>()) : f(t, d, std::integral_constant<int, 2>());
    };
    using D64 = std::integral_constant<int, 64>;
    using D128 = std::integral_constant<int, 128>;
    if (type == ElemType::kBF16) return dim == 64 ? by_rows(__nv_bfloat16(), D64()) : by_rows(__nv_bfloat16(), D128());
    return dim == 64 ? by_rows(__half(), D64()) : by_rows(__half(), D128());
}

}  // namespace

LIBGEMM_DEBUG_READER(kv4_attention_debug_flags)

cudaError_t kv4_attention_setup() {
    for (ElemType type : {ElemType::kBF16, ElemType::kF16})
        for (int dim : {64, 128})
            for (int rows : {8, 16}) {
                const cudaError_t e = with_kernel(type, dim, rows, [](auto t, auto d, auto nq) {
                    constexpr int D = decltype(d)::value, NQ = decltype(nq)::value;
                    return cudaFuncSetAttribute(kv4_attention_kernel<decltype(t), D, NQ>,
                                                cudaFuncAttributeMaxDynamicSharedMemorySize, Ring<D, NQ>::kBytes);
                });
                if (e != cudaSuccess) return e;
            }
    return cudaSuccess;
}

cudaError_t launch_kv4_few(const AttnArgs& a, ElemType type, const KvPlan& plan, cudaStream_t stream) {
    return with_kernel(type, a.c.dim, plan.rows, [&](auto t, auto d, auto nq) {
        return launch<decltype(t), decltype(d)::value, decltype(nq)::value>(a, plan, stream);
    });
}

}  // namespace libgemm
