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
// rounded, so that their rounding errors meet c and not u.  It does so in every step
// of 32 tokens: taken out once at the end, the sums of u and of 8, which the matrix
// instruction truncates, were off by 0.4 % of the results' size over 32768 tokens of
// one warp's four and by 7 % over 200001 (now under 0.01 %), for 1.5 % of the time.
//
// Every token has its own scales.  A page and head's codes and scales lie in one
// piece, and one bulk copy brings them.
//
// Weights, times their token's value scale, are binary16 in the second product: with
// more bits it would have to be made twice.  Results are 1.74e-3 of their size from 64
// bits in bfloat16 and 2.9e-4 in binary16, where rounding them is 1.73e-3 and 2.1e-4
// (8192 tokens, normal queries and values).
//
// 64 sequences of up to 8192 tokens, 64 heads over 8 of 128: 318 MB in 67.5 us, 4.7
// TB/s or 69 % of the measured copy rate (over 8 bits 617 MB in 123 us).  Between a
// CTA's first stage and its last that is 6.3 TB/s; the rest is its beginning (6.5 us:
// 2.1 to find its piece, 2.3 to look its tile and queries up, 2 for the first copies,
// which all ask for at once), the parting of the CTAs' ends (57 to 64 us) and the
// joining launch (2.8).  Up to 32768 tokens take 214 us, 88 %.  A warp had 212
// instructions for 16 tokens, 117 of them on the ALU pipe, before the 8 of the codes
// came off in every step, for which 8 more (66.5 us then, and 211).
// Tiles of 16 rows, two CTAs an SM: the same with two queries a sequence takes 145 us.
// Three CTAs an SM, as 128 registers allow, of four computing warps and a copying
// one each.  With two an SM, and a cluster a tile, 110 us; with three, and sums that
// change their reference seldom, 92; all steps in one line 82, flags of the stages
// that every row sees whole 80, tiles' openings counted 70, results joined four at a
// time 67.5.  Left: four CTAs an SM without a copying warp 108 (when it was 92), or
// with 96 registers 97 (78); two or three times as many pieces 94 and 100 (93);
// values' codes loaded before the weights are made 83 (82); the first copies before
// the queries 69 (67.5: the queries wait behind them).
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

// A bfloat16 in shared memory.
__device__ __forceinline__ float lds_bf16(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
    return __uint_as_float((uint32_t)v << 16);
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
constexpr uint32_t kPlain = 256;
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

// The ring's place in shared memory, and where a warp is in its rounds.
template <int D, int NQ>
struct Stages {
    using R = Ring<D, NQ>;
    uint32_t ring, bars;            // full[stages], empty[stages]
    uint32_t* live_subs;            // which 16s of a stage are there; kPlain: all, and every row sees all of them
    volatile int* abort_flag;
    uint32_t phase = 0;
    int stage = 0;
    __device__ __forceinline__ explicit Stages(uint8_t* smem)
        : ring(smem_u32(smem)), bars(ring + R::kBarsAt), live_subs(reinterpret_cast<uint32_t*>(smem + R::kLiveAt)),
          abort_flag(reinterpret_cast<volatile int*>(smem + R::kAbortAt)) {}
    __device__ __forceinline__ void init() const {   // one thread
        for (int s = 0; s < R::kStages; ++s) {
            mbar_init(bars + 8 * s, 1);
            mbar_init(bars + 8 * (R::kStages + s), kWarps);
        }
        *abort_flag = 0;
        mbar_fence_init();
    }
    __device__ __forceinline__ uint32_t at() const { return ring + stage * R::kStageBytes; }
    __device__ __forceinline__ bool wait_full(unsigned* err) const { return warp_wait(bars + 8 * stage, phase, abort_flag, err); }
    __device__ __forceinline__ bool wait_empty(unsigned* err) const { return warp_wait(bars + 8 * (R::kStages + stage), phase ^ 1u, abort_flag, err); }
    __device__ __forceinline__ void release() { warp_arrive(bars + 8 * (R::kStages + stage)); }
    __device__ __forceinline__ void next() {
        if (++stage == R::kStages) stage = 0, phase ^= 1u;
    }
};

// The copying warp: `steps` stages of a tile's tokens from tok_begin on.  Lane i
// looks up 16 tokens, those of four stages at a time.  False if a wait gave up.
template <int D, int NQ>
__device__ __forceinline__ bool copy_steps(const AttnArgs& a, const Tile& tile, int h, int tok_begin, int steps, Stages<D, NQ>& st, int& issued) {
    static_assert(kWarps * kSubs == 8, "");
    const int lane = threadIdx.x % 32, log2 = a.c.page_log2, record = (D + 4) << log2;
    const int32_t* table = a.b.table + tile.seq * a.b.width;
    [[maybe_unused]] const int64_t extent = a.c.pages * a.c.heads * a.c.record();
    // tokens that every row of the tile sees
    const int full_lo = tile.row_lo(a, min(tile.r0 + 8 * NQ, tile.nrows) - 1), full_hi = tile.row_hi(a, tile.r0);
    bool live = false;
    const uint8_t* from = nullptr;
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
        if (!st.wait_empty(a.err)) return false;
        const int sub = lane - s % 4 * 8;   // this lane's part of the stage, if it has one
        const bool here = sub >= 0 && sub < 8 && live;
        bool copies = here && (sub * kSub & ((1 << log2) - 1)) == 0;   // a page's first 16 tokens fetch all of it
        if (copies) copies = GEMM_DBG_OK(from, a.c.data, extent, record);
        const unsigned there = __ballot_sync(0xFFFFFFFFu, here), parts = __popc(__ballot_sync(0xFFFFFFFFu, copies));
        if (copies) bulk_load(st.at() + (sub * kSub >> log2) * record, from, record, st.bars + 8 * st.stage);
        __syncwarp();
        if (lane == 0) {
            const int tok = tok_begin + s * kStep;
            const uint32_t subs = there >> (s % 4 * 8);
            st.live_subs[st.stage] = subs == 255u && tok >= full_lo && tok + kStep <= full_hi ? subs | kPlain : subs;
            mbar_arrive_expect_tx(st.bars + 8 * st.stage, parts * record);
        }
        ++issued;
        st.next();
    }
    return true;
}
// Copies in flight land before the CTA may leave or reuse the ring.
template <int D, int NQ>
__device__ __forceinline__ void drain_all(const Stages<D, NQ>& st, int issued, unsigned* err) {
    constexpr int kStages = Ring<D, NQ>::kStages;
    if (threadIdx.x % 32 == 0)
        for (int s = max(0, issued - kStages); s < issued; ++s) drain(st.bars + 8 * (s % kStages), (uint32_t)(s / kStages) & 1u, err);
    __syncwarp();
}

// Elements d .. d + 7 of a tile's row r, 0 past the last row.
template <typename T, int D>
__device__ __forceinline__ Eight<T> query(const AttnArgs& a, const Tile& tile, int h, int r, int d) {
    [[maybe_unused]] const int64_t q_bytes = ((a.b.rows - 1) * a.Q.row + (a.q_heads - 1) * a.Q.head + D) * (int64_t)sizeof(T);
    const unsigned row = tile.r0 + r;
    Eight<T> x = {};
    if (row >= (unsigned)tile.nrows) return x;
    const T* p = static_cast<const T*>(a.Q.p) + (int64_t)(tile.row0 + row / a.share) * a.Q.row + (int64_t)(h * a.share + row % a.share) * a.Q.head + d;
    if (GEMM_DBG_OK(p, a.Q.p, q_bytes, 16)) x = load_eight(p, a.q_vec);
    return x;
}

// One warp's part of a tile of 8 * NQ rows: the tokens' side is the 16-row operand
// of both products and the queries its eight columns: S^T = K Q^T, then O^T = V^T
// P^T, for which the weights are turned over in registers.
template <typename T, int D, int NQ>
struct Attend {
    static constexpr int kLd = D + 4, kWords = D / 32;
    static constexpr int MT = D / 16;   // row tiles of O^T: row g of tile 2i + x is d = 64 (i / 2) + 8g + 4 (i % 2) + 2x, row g + 8 the next
    // Query row 8n + g as the column g of B.  A lane's part of a row is 8
    // neighbours of each 32: elements e and e + 4 a word's two halves hold
    // together.  Rows are brought to [2^11, 2^12) by a power of two, so that 16
    // times that is binary16 (exact, but for elements under 2^-25 of the row's
    // largest, whose error stays under 2^-36 of it).
    uint32_t qf[NQ][2 * kWords][2];
    float factor[NQ][2], begin[NQ][4];      // of the rows 8n + 2t, + 1, whose scores a lane gets
    int row_lo[NQ][2], row_hi[NQ][2];
    // A row's sums: l of the weights exp2(s_j - m) in binary32, o of the codes times
    // those times their token's value scale v_j times up = 2^12 / r as binary16, where
    // m and r are the row's own largest s_j and exp2(s_j - m) * v_j so far, of tokens
    // that it sees (r at least kLeastP).
    float o[NQ][MT][4], m[NQ][2], l[NQ][2], up[NQ][2];

    // get(r, d): elements d .. d + 7 of the tile's row r, 0 past its last.
    template <typename F>
    __device__ __forceinline__ void start(const AttnArgs& a, const Tile& tile, F get) {
        const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            Eight<T> x[kWords];
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < kWords; ++i) x[i] = get(8 * n + g, 32 * i + 8 * t);
#pragma unroll
            for (int i = 0; i < kWords; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[i].at(e)));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            // its biased exponent, in the range in which the powers below, and 16 times the
            // first, are finite and normal: rows of zeros stay zeros
            const int k = top < INFINITY ? max(15, (int)(__float_as_uint(top) >> 23)) : 127;
            const float down = __uint_as_float((uint32_t)(265 - k) << 23) * (a.scale_log2 < 0.0f ? -1.0f : 1.0f);   // 2^(11 + 127 - k)
            const float back = __uint_as_float((uint32_t)k << 23);   // 2^(k - 127); 2^9 more for the 2^-11 above and the codes' 2^-20
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
                // above 0, so that a hidden token's -inf stays that, and finite
                factor[n][i] = fminf(fmaxf(fabsf(a.scale_log2) * 512.0f * __shfl_sync(0xFFFFFFFFu, back, 4 * (2 * t + i)), 1.1754943508222875e-38f), 3.4028235e38f);
                // rows past the last one see all: they are not stored
                const int rr = tile.r0 + 8 * n + 2 * t + i;
                row_lo[n][i] = rr < tile.nrows ? tile.row_lo(a, rr) : 0;
                row_hi[n][i] = rr < tile.nrows ? tile.row_hi(a, rr) : tile.hi;
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.0f;
            m[n][0] = m[n][1] = kLowest;
            l[n][0] = l[n][1] = 0.0f;
            up[n][0] = up[n][1] = kTopP / kLeastP;
        }
    }

    // Where this warp's tokens lie in every stage: the keys' codes of token g of its
    // first 16 and the values' piece of this lane, the key scale of that token, what
    // the second 16 are further on, and what value scales are behind key scales.
    uint32_t key_at, value_at, scale_at, next_codes, next_scales, to_values;
    __device__ __forceinline__ void locate(int log2) {
        const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
        const int page_tokens = 1 << log2, record = (D + 4) << log2, at = warp * (kSubs * kSub);
        const uint32_t page = (at >> log2) * record, in = at & (page_tokens - 1);
        key_at = page + in * (D / 2) + g * (D / 2) + t * (D / 8);
        value_at = page + (page_tokens + in) * (D / 2) + lane * (D / 8);
        scale_at = page + page_tokens * D + 2 * (in + g);
        next_codes = log2 == 4 ? record : kSub * (D / 2);
        next_scales = log2 == 4 ? record : 2 * kSub;
        to_values = 2 * page_tokens;
    }

    // This warp's 32 tokens of a stage, from token `tok` on; `subs`: which 16s are
    // there.  `masked`: of some that some row does not see, or that are not there.
    __device__ __forceinline__ void step(uint32_t stage_at, int tok, uint32_t subs, bool masked) {
        const int lane = threadIdx.x % 32, g = lane / 4;
        // scores of tokens 16b + g and 16b + g + 8 (y) for the rows 2t (.x) and 2t + 1 (.y)
        float2 sc[kSubs][NQ][2];
        float vs[kSubs][2];
#pragma unroll
        for (int b = 0; b < kSubs; ++b) {
            const uint32_t kat = stage_at + key_at + b * next_codes, sat = stage_at + scale_at + b * next_scales;
            uint32_t w0[kWords], w1[kWords];
            load_words<D>(kat, w0);
            load_words<D>(kat + 8 * (D / 2), w1);
            const float ks[2] = {lds_bf16(sat), lds_bf16(sat + 16)};
            vs[b][0] = lds_bf16(sat + to_values), vs[b][1] = lds_bf16(sat + to_values + 16);
            float part[NQ][4];
#pragma unroll
            for (int i = 0; i < kWords; ++i)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t lo = w0[i] >> (8 * x), hi = w1[i] >> (8 * x);
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
                        mma_16816_from(part[n], i + x > 0 ? part[n] : begin[n], lo & kLow, hi & kLow, lo & kHigh, hi & kHigh, qf[n][2 * i + x][0],
                                       qf[n][2 * i + x][1]);
                }
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int y = 0; y < 2; ++y)
                    sc[b][n][y] = __fmul2_rn(make_float2(part[n][2 * y], part[n][2 * y + 1]), make_float2(ks[y], ks[y]));
        }
        // Tokens that some row does not see, pages that do not exist.  There a weight
        // of 0 has to stay 0 whatever the token has for a scale, and a scale of NaN
        // makes NaN of the rows alone that see it; elsewhere all rows see all tokens.
        uint32_t nan = 0;
        if (masked) {
#pragma unroll
            for (int b = 0; b < kSubs; ++b)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int j = tok + 16 * b + g + 8 * y;
                    const bool live = subs >> b & 1u;
#pragma unroll
                    for (int n = 0; n < NQ; ++n) {
                        if (j < row_lo[n][0] || j >= row_hi[n][0] || !live) sc[b][n][y].x = kNegInf;
                        if (j < row_lo[n][1] || j >= row_hi[n][1] || !live) sc[b][n][y].y = kNegInf;
                    }
                    if (vs[b][y] != vs[b][y]) nan |= 1u << (2 * b + y);
                    vs[b][y] = fminf(fabsf(vs[b][y]), 3.3895314e38f);
                }
        }
        // A weight, and it with its token's value scale, relative to the row's largest.
        float2 w[kSubs][NQ][2], p[kSubs][NQ][2];
        auto weigh = [&] {   // returns the largest weight of either product
            float most = 0.0f;
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                const float2 f = make_float2(factor[n][0], factor[n][1]), less = make_float2(-m[n][0], -m[n][1]), u = make_float2(up[n][0], up[n][1]);
#pragma unroll
                for (int b = 0; b < kSubs; ++b)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float2 x = __ffma2_rn(sc[b][n][y], f, less);
                        const float2 e = make_float2(exp2_approx(x.x), exp2_approx(x.y));
                        const float2 v = __fmul2_rn(__fmul2_rn(e, u), make_float2(vs[b][y], vs[b][y]));   // (0 of a weight of 0)
                        w[b][n][y] = e, p[b][n][y] = v;
                        most = max3(max3(most, e.x, v.x), e.y, v.y);
                    }
            }
            return most;
        };
        // A row's sums so far are brought to a new maximum only when it is passed
        // by so much that a weight might not fit binary16, whatever the other
        // rows do: a row's result does not depend on its neighbours.
        if (__any_sync(0xFFFFFFFFu, weigh() > kMostP)) {
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                float grow[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    auto of = [&](const float2& x) { return i ? x.y : x.x; };
                    auto across = [](float x) {   // the largest of the lanes that have this row
                        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
                        return fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
                    };
                    float most = 0.0f, highest = kNegInf;
#pragma unroll
                    for (int b = 0; b < kSubs; ++b)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            most = max3(most, of(w[b][n][y]), of(p[b][n][y]));
                            highest = fmaxf(highest, of(sc[b][n][y]));
                        }
                    // (every lane takes part in every exchange, also those whose row stays)
                    const bool passed = across(most) > kMostP;
                    highest = across(highest * factor[n][i]);
                    const float top = passed ? fmaxf(highest, m[n][i]) : m[n][i];
                    const float keep = exp2_approx(m[n][i] - top), sums = keep * __fdividef(kTopP, up[n][i]);
                    m[n][i] = top;
                    l[n][i] *= keep;
                    float rel = 0.0f;
#pragma unroll
                    for (int b = 0; b < kSubs; ++b)
#pragma unroll
                        for (int y = 0; y < 2; ++y) rel = fmaxf(rel, exp2_approx(fmaf(of(sc[b][n][y]), factor[n][i], -top)) * vs[b][y]);
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
            }
            weigh();
        }
        if (masked && __any_sync(0xFFFFFFFFu, nan != 0)) {
            const float bad = __uint_as_float(0x7FC00000u);
#pragma unroll
            for (int b = 0; b < kSubs; ++b)
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        if (nan >> (2 * b + y) & 1u)
                            p[b][n][y] = make_float2(sc[b][n][y].x == kNegInf ? 0.0f : bad, sc[b][n][y].y == kNegInf ? 0.0f : bad);
        }
        float ones[NQ][4] = {};   // sums of the weights as they enter the product: rows all alike
#pragma unroll
        for (int b = 0; b < kSubs; ++b) {
            const uint32_t vat = stage_at + value_at + b * next_codes;
            uint32_t w0[kWords], w1[kWords];   // tokens 2t, 2t + 1; those 8 on
            load_words<D>(vat, w0);
            load_words<D>(vat + 4 * D, w1);
            // Binary16 under 2^16, normal down to 2^-26 of the row's largest.
            uint32_t pt[NQ][2];
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                const float2 sum = __fadd2_rn(__fadd2_rn(w[b][n][0], w[b][n][1]), make_float2(l[n][0], l[n][1]));
                l[n][0] = sum.x, l[n][1] = sum.y;
                pt[n][0] = transpose8(pack2<__half>(p[b][n][0].x, p[b][n][0].y));
                pt[n][1] = transpose8(pack2<__half>(p[b][n][1].x, p[b][n][1].y));
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
        // The codes' 8 comes off here, not at the end: the matrix instruction's sums lose
        // up to a last place towards 0 each, of all that they have so far, and 8 times
        // the weights would outgrow the results by the root of the tokens' number.
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const float2 high = __fmul2_rn(make_float2(ones[n][0], ones[n][1]), make_float2(-8.0f * 9.5367431640625e-7f, -8.0f * 9.5367431640625e-7f));   // 2^-20
            const float2 low = __fmul2_rn(high, make_float2(0.0625f, 0.0625f));
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const float2 x = __fadd2_rn(make_float2(o[n][i][0], o[n][i][1]), low), y = __fadd2_rn(make_float2(o[n][i][2], o[n][i][3]), high);
                o[n][i][0] = x.x, o[n][i][1] = x.y, o[n][i][2] = y.x, o[n][i][3] = y.y;
            }
        }
    }

    // The sums of rows 8n .. 8n + 7 into s_o[warp][8][kLd], s_m and s_l[warp][8].
    __device__ __forceinline__ void put(int n, float* s_o, float* s_m, float* s_l) {
        const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int at = warp * 8 + 2 * t + i;
            const float unit = 1.0f / up[n][i];
            l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], 4);
            l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], 8);
            l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], 16);
            if (g == 0) s_m[at] = m[n][i], s_l[at] = l[n][i];
#pragma unroll
            for (int e = 0; e < kWords; ++e) {
                auto value = [&](int x, int row) { return o[n][2 * e + x][2 * row + i] * (row ? 1048576.0f : 16777216.0f) * unit; };   // 2^20, 2^24
                *reinterpret_cast<float4*>(s_o + at * kLd + 64 * (e / 2) + 8 * g + 4 * (e % 2)) =
                    make_float4(value(0, 0), value(0, 1), value(1, 0), value(1, 1));
            }
        }
    }
    // Elements d .. d + 3 of row r (0 .. 7) of what the warps have put: maximum, sum of weights, results so far.
    static __device__ __forceinline__ void joined(const float* s_o, const float* s_m, const float* s_l, int r, int d, float& top, float& sum, float4& acc) {
        top = s_m[r];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_m[w * 8 + r]);
        sum = 0.0f;
        acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = exp2_approx(s_m[w * 8 + r] - top);
            const float4 x = *reinterpret_cast<const float4*>(s_o + (w * 8 + r) * kLd + d);
            sum = fmaf(f, s_l[w * 8 + r], sum);
            acc.x = fmaf(f, x.x, acc.x), acc.y = fmaf(f, x.y, acc.y), acc.z = fmaf(f, x.z, acc.z), acc.w = fmaf(f, x.w, acc.w);
        }
    }
    static __device__ __forceinline__ void store(T* to, const float4& acc, float sum) {
        const float x[4] = {acc.x, acc.y, acc.z, acc.w};
        uint32_t y[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) y[i] = pack2<T>(sum == 0.0f ? 0.0f : x[2 * i] / sum, sum == 0.0f ? 0.0f : x[2 * i + 1] / sum);
        if ((reinterpret_cast<uintptr_t>(to) & 7u) == 0) {
            *reinterpret_cast<uint2*>(to) = make_uint2(y[0], y[1]);
        } else {
            const T* e = reinterpret_cast<const T*>(y);
            to[0] = e[0], to[1] = e[1], to[2] = e[2], to[3] = e[3];
        }
    }
};

// Few tiles: one of 8 * NQ rows over a share of its tokens for each CTA, and a
// tile's CTAs a cluster, which joins through distributed shared memory.  One warp
// copies pages into a ring of stages of 128 tokens, four take 32 tokens of each.
template <typename T, int D, int NQ>
__global__ void __launch_bounds__(kThreads, resident(NQ)) kv4_cluster_kernel(const AttnArgs a) {
    using R = Ring<D, NQ>;
    using A = Attend<T, D, NQ>;
    constexpr int kRows = 8 * NQ, kGroup = kWarps * 8 * A::kLd;   // floats of eight rows
    static_assert(NQ * kGroup * 4 + (2 * kWarps + 2) * kRows * 4 <= R::kLiveAt, "the joining reuses the ring");
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x / 32;
    const int u = blockIdx.x / a.splits, split = blockIdx.x % a.splits, h = blockIdx.y;
    Tile tile;
    // A cluster's CTAs have one tile: they leave here together or not at all.
    if (!tile.find(a, u, kRows, kStep, h == 0 && split == 0)) return;
    const int step_begin = min(tile.steps, split * tile.per);
    const int steps = min(tile.steps, step_begin + tile.per) - step_begin;
    const int tok_begin = tile.tok0 + step_begin * kStep;
    Stages<D, NQ> st(smem);
    if (threadIdx.x == 0) st.init();
    __syncthreads();

    float* s_o = reinterpret_cast<float*>(smem);     // [NQ][warps][8][kLd]
    float* s_m = s_o + NQ * kGroup;                  // [NQ][warps][8]
    float* s_l = s_m + kWarps * kRows;
    float* s_joined = s_l + kWarps * kRows;          // (maximum, sum) of each row
    if (warp == kWarps) {
        int issued = 0;
        copy_steps(a, tile, h, tok_begin, steps, st, issued);
        drain_all(st, issued, a.err);
        __syncthreads();   // the ring is free
        __syncthreads();   // the warps' results are in it
    } else {
        A rows;
        rows.locate(a.c.page_log2);
        rows.start(a, tile, [&](int r, int d) { return query<T, D>(a, tile, h, r, d); });
        for (int s = 0; s < steps; ++s) {
            if (!st.wait_full(a.err)) break;
            const uint32_t subs = st.live_subs[st.stage];
            const int tok = tok_begin + s * kStep + warp * (kSubs * kSub);
            if (tok < tile.hi) rows.step(st.at(), tok, subs >> (warp * kSubs), !(subs & kPlain));
            st.release();
            st.next();
        }
        __syncthreads();   // the ring is free: every copy has landed and been used
#pragma unroll
        for (int n = 0; n < NQ; ++n) rows.put(n, s_o + n * kGroup, s_m + n * kWarps * 8, s_l + n * kWarps * 8);
        __syncthreads();
    }

    [[maybe_unused]] const int64_t o_bytes =
        ((a.b.rows - 1) * a.O.row + (a.q_heads - 1) * a.O.head + D) * (int64_t)sizeof(T);
    const int rows = min(tile.nrows - tile.r0, kRows);
    auto place = [&](int r, int d) { return s_o + r / 8 * kGroup + r % 8 * A::kLd + d; };   // warp 0's
    for (int i = 4 * threadIdx.x; i < rows * D; i += 4 * kThreads) {
        const int r = i / D, d = i % D;
        float top, sum;
        float4 acc;
        A::joined(s_o + r / 8 * kGroup, s_m + r / 8 * kWarps * 8, s_l + r / 8 * kWarps * 8, r % 8, d, top, sum, acc);
        if (a.splits == 1) {
            T* dst = out_row<T>(a, tile, h, tile.r0 + r) + d;
            if (GEMM_DBG_OK(dst, a.O.p, o_bytes, 4 * sizeof(T))) A::store(dst, acc, sum);
        } else {
            *reinterpret_cast<float4*>(place(r, d)) = acc;   // read by this thread alone so far
            if (d == 0) s_joined[2 * r] = top, s_joined[2 * r + 1] = sum;
        }
    }
    if (a.splits == 1) return;
    // The cluster's CTAs each join a share of the results, in split order.
    cluster_sync();
    const int share = (rows * D + a.splits - 1) / a.splits;
    for (int i = split * share + threadIdx.x; i < min(rows * D, (split + 1) * share); i += kThreads) {
        const int r = i / D, d = i % D;
        const uint32_t ml = smem_u32(s_joined + 2 * r), at = smem_u32(place(r, d));
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

// ---- many tiles ------------------------------------------------------------------
// All steps of all tiles and heads stand in one line, sequences first, then tiles,
// heads and steps, and each CTA of one round takes an equal piece of it: its first
// and its last tile may be others' too, and a second launch joins those.  (A
// sequence's tiles count as many steps each as its longest can have: a walk needs
// lengths and row counts alone.)  What a tile's beginning and end take counts as
// kOpening steps at its head; where a piece would begin or end among these, it
// does so before them.
constexpr int kOpening = 3;   // 8192 tokens: 2 69.8 us, 3 67.5, 4 67.5, 5 69.4; 0 78
struct Walk {
    int seq;
    int64_t at, left;                  // place among the sequence's steps; steps still to go
    int row0, count, len, tiles;
    int64_t weight;                    // steps of each of its tiles and heads, and kOpening

    // Sequence q's numbers; `report`: one thread of the launch says what is out of range.
    __device__ __forceinline__ void look(const AttnArgs& a, int q, int rows, bool report) {
        const Starts starts{a.b.starts, a.b.sequences, a.b.rows};
        seq = q;
        row0 = (int)starts.at(q);
        const bool good = starts.good(q);
        count = good ? (int)starts.at(q + 1) - row0 : 0;
        len = __ldg(a.b.at + q);
        if (count > 0 && (len < 0 || len > (a.b.width << a.c.page_log2))) {
            if (report) atomicOr(a.err, kErrIndex);
            len = 0;
        }
        if (!good && report) atomicOr(a.err, kErrIndex);
        tiles = (int)(((int64_t)count * a.share + rows - 1) / rows);
        weight = ((int64_t)len + kStep - 1) / kStep;
        if (a.window > 0) {   // the window, the tile's positions, and a step's beginning
            const int64_t seen = ((int64_t)a.window + rows / a.share + 1 + 2 * (kStep - 1)) / kStep;
            weight = weight < seen ? weight : seen;
        }
        weight = (weight < 1 ? 1 : weight) + kOpening;
    }
    __device__ __forceinline__ int64_t steps(const AttnArgs& a) const { return (int64_t)tiles * a.c.heads * weight; }
};

// A CTA's next part of one tile and head, as the copying warp tells it the others
// at the head of a stage, the queries behind it.
struct alignas(16) Piece {
    Tile tile;
    int h, begin, steps;
    bool first, whole, end;              // it has the tile's first token, all of them; end: there is none
};

// False at the end.
__device__ __forceinline__ bool next_piece(const AttnArgs& a, Walk& w, int rows, Piece& piece) {
    Tile& tile = piece.tile;
    if (w.left <= 0) return false;
    while (w.at >= w.steps(a)) {
        w.at -= w.steps(a);
        if (w.seq + 1 >= a.b.sequences) return false;
        w.look(a, w.seq + 1, rows, false);
    }
    const int64_t which = w.at / w.weight, k = w.at - which * w.weight;
    const int j = (int)(which / a.c.heads);
    const int64_t n = w.weight - k < w.left ? w.weight - k : w.left;
    if (k == 0 && n <= kOpening) return false;   // the next CTA's
    const int64_t begin = k == 0 ? 0 : k - kOpening, end = k + n - kOpening;
    piece.h = (int)(which - (int64_t)j * a.c.heads);
    tile.place(a, w.seq, w.row0, w.count, w.len, j * rows, rows, kStep);
    piece.begin = (int)(begin < tile.steps ? begin : tile.steps);
    piece.steps = (int)(end < tile.steps ? end : tile.steps) - piece.begin;
    piece.first = k == 0;
    piece.whole = k == 0 && n == w.weight;
    w.at += n;
    w.left -= n;
    return true;
}

// A barrier of the four warps that compute, and whether all of them are `well`.
__device__ __forceinline__ bool warps_agree(bool well) {
    uint32_t all;
    asm volatile(
        "{\n"
        ".reg .pred p, q;\n"
        "setp.ne.u32 q, %1, 0;\n"
        "bar.red.and.pred p, 1, %2, q;\n"
        "selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(all)
        : "r"((uint32_t)well), "n"(kWarps * 32)
        : "memory");
    return all != 0;
}

template <typename T, int D, int NQ>
__global__ void __launch_bounds__(kThreads, resident(NQ)) kv4_line_kernel(const AttnArgs a) {
    using R = Ring<D, NQ>;
    using A = Attend<T, D, NQ>;
    constexpr int kRows = 8 * NQ;
    static_assert(kWarps * 8 * A::kLd * 4 <= R::kStageBytes && sizeof(Piece) + kRows * D * 2 <= R::kStageBytes && R::kStageBytes % 16 == 0 && NQ <= R::kStages,
                  "eight rows of four warps fit a stage, and a piece with its queries");
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t s_sum[kThreads / 32];
    __shared__ Walk s_walk;
    __shared__ float s_ml[2][2][NQ][kWarps * 8];     // of a piece and of the next: maxima, sums
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    grid_launch_dependents();   // the joining launch may start its set-up
    Stages<D, NQ> st(smem);
    if (threadIdx.x == 0) st.init();
    if (blockIdx.x == 0) Starts{a.b.starts, a.b.sequences, a.b.rows}.check(a.err);

    // Where this CTA's piece of the line begins: sums over sequences, a thread
    // some neighbours, then the thread that has the beginning looks for it.
    const int each = (a.b.sequences + kThreads - 1) / kThreads, q0 = min(a.b.sequences, (int)threadIdx.x * each), q1 = min(a.b.sequences, q0 + each);
    Walk walk;
    int64_t mine = 0;
    for (int q = q0; q < q1; ++q) {
        walk.look(a, q, kRows, blockIdx.x == 0);
        mine += walk.steps(a);
    }
    int64_t before = mine;
    for (int i = 1; i < 32; i *= 2) {
        const int64_t x = __shfl_up_sync(0xFFFFFFFFu, before, i);
        if (lane >= i) before += x;
    }
    if (lane == 31) s_sum[warp] = before;
    if (threadIdx.x == 0) s_walk.seq = -1;
    __syncthreads();
    int64_t all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w == warp) before += all;
        all += s_sum[w];
    }
    before -= mine;
    const int64_t per = (all + gridDim.x - 1) / gridDim.x, lo = per * blockIdx.x;
    if (mine > 0 && before <= lo && lo < before + mine) {
        int64_t at = lo - before;
        for (int q = q0; q < q1; ++q) {
            walk.look(a, q, kRows, false);
            if (at < walk.steps(a)) break;
            at -= walk.steps(a);
        }
        const int64_t k = at % walk.weight, back = k <= kOpening ? k : 0;
        walk.at = at - back;
        walk.left = (per < all - lo ? per : all - lo) + back;
        s_walk = walk;
    }
    __syncthreads();
    if (s_walk.seq < 0) return;   // past the end of the line
    walk = s_walk;

    if (warp == kWarps) {
        int issued = 0;
        Piece piece;
        for (bool ok = true; ok;) {
            piece.end = !next_piece(a, walk, kRows, piece);
            if (!(ok = st.wait_empty(a.err))) break;
            uint8_t* at = smem + st.stage * R::kStageBytes;
            if (lane == 0) *reinterpret_cast<Piece*>(at) = piece;
            if (!piece.end) {
                Eight<T> x[kRows * D / 256];
#pragma unroll
                for (int i = 0; i < kRows * D / 256; ++i) x[i] = query<T, D>(a, piece.tile, piece.h, (i * 32 + lane) / (D / 8), (i * 32 + lane) % (D / 8) * 8);
#pragma unroll
                for (int i = 0; i < kRows * D / 256; ++i) *reinterpret_cast<uint4*>(at + sizeof(Piece) + 16 * (i * 32 + lane)) = x[i].v[0];
            }
            auto pass = [&] {
                __syncwarp();
                if (lane == 0) mbar_arrive(st.bars + 8 * st.stage);
                ++issued;
                st.next();
            };
            pass();
            if (piece.end) break;
            ok = copy_steps(a, piece.tile, piece.h, piece.tile.tok0 + piece.begin * kStep, piece.steps, st, issued);
            for (int n = 0; ok && n < NQ; ++n) {   // stages for the warps to join in
                if ((ok = st.wait_empty(a.err))) pass();
            }
        }
        drain_all(st, issued, a.err);
        return;
    }
    [[maybe_unused]] const int64_t o_bytes =
        ((a.b.rows - 1) * a.O.row + (a.q_heads - 1) * a.O.head + D) * (int64_t)sizeof(T);
    A rows;
    rows.locate(a.c.page_log2);
    bool ok = true;   // of all four warps alike, from one joining to the next
    for (int turn = 0; ok; turn ^= 1) {
        if (!(ok = warps_agree(st.wait_full(a.err)))) break;
        const uint8_t* at = smem + st.stage * R::kStageBytes;
        const Piece piece = *reinterpret_cast<const Piece*>(at);
        if (piece.end) break;
        const Tile& tile = piece.tile;
        rows.start(a, tile, [&](int r, int d) {
            Eight<T> x;
            x.v[0] = *reinterpret_cast<const uint4*>(at + sizeof(Piece) + (r * D + d) * 2);
            return x;
        });
        fence_proxy_async_shared();   // copies into this stage come after
        st.release();
        st.next();
        const int tok_begin = tile.tok0 + piece.begin * kStep;
        for (int s = 0; ok && s < piece.steps; ++s) {
            if (!(ok = st.wait_full(a.err))) break;
            const uint32_t subs = st.live_subs[st.stage];
            const int tok = tok_begin + s * kStep + warp * (kSubs * kSub);
            if (tok < tile.hi) rows.step(st.at(), tok, subs >> (warp * kSubs), !(subs & kPlain));
            st.release();
            st.next();
        }
        // A slot for the tile that others began, one for that which others go on with.
        float* slot = a.partial + ((int64_t)blockIdx.x * 2 + (piece.first ? 1 : 0)) * (kRows * (D + 2));
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            ok = ok && st.wait_full(a.err);
            float* s_o = reinterpret_cast<float*>(smem + st.stage * R::kStageBytes);
            float *s_m = s_ml[turn][0][n], *s_l = s_ml[turn][1][n];
            if (ok) rows.put(n, s_o, s_m, s_l);
            if (!(ok = warps_agree(ok))) break;
            const int live = min(tile.nrows - tile.r0 - 8 * n, 8);
            for (int i = 4 * threadIdx.x; i < live * D; i += 4 * kWarps * 32) {
                const int r = i / D, d = i % D;
                float top, sum;
                float4 acc;
                A::joined(s_o, s_m, s_l, r, d, top, sum, acc);
                if (piece.whole) {
                    T* dst = out_row<T>(a, tile, piece.h, tile.r0 + 8 * n + r) + d;
                    if (GEMM_DBG_OK(dst, a.O.p, o_bytes, 4 * sizeof(T))) A::store(dst, acc, sum);
                } else {
                    float *to = slot + (8 * n + r) * D + d, *ml = slot + kRows * D + 2 * (8 * n + r);
                    if (GEMM_DBG_OK(to, a.partial, a.partial_bytes, 16)) *reinterpret_cast<float4*>(to) = acc;
                    if (d == 0 && GEMM_DBG_OK(ml, a.partial, a.partial_bytes, 8)) ml[0] = top, ml[1] = sum;
                }
            }
            fence_proxy_async_shared();   // copies into this stage come after
            st.release();
            st.next();
        }
    }
}

// Joins the tiles that were shared, in the order of their tokens: a warp a row
// (TEAM = 1), or eight warps one where few tiles are shared by many CTAs each, so that
// all parts' loads are under way at once.  Which CTAs have a tile follows from the
// lengths, and is found before the parts are there.
template <typename T, int D, int NQ, int TEAM>
__global__ void __launch_bounds__(256) kv4_line_join_kernel(const AttnArgs a) {
    constexpr int kRows = 8 * NQ, kEach = D / 32, kBatch = 4;
    __shared__ float s_acc[TEAM][D], s_sum[TEAM];
    __shared__ int64_t s_before[8], s_all[8];
    const int u = blockIdx.x, h = blockIdx.y, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    Tile tile;
    if (!tile.find(a, u, kRows, kStep, false)) {
        grid_dependency_wait();   // this launch does not end before the one that makes the parts
        return;
    }
    int64_t before = 0, all = 0;
    Walk walk;
    for (int q = threadIdx.x; q < a.b.sequences; q += 256) {
        walk.look(a, q, kRows, false);
        const int64_t steps = walk.steps(a);
        all += steps;
        if (q < tile.seq) before += steps;
    }
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) {
        before += __shfl_xor_sync(0xFFFFFFFFu, before, i);
        all += __shfl_xor_sync(0xFFFFFFFFu, all, i);
    }
    if (lane == 0) s_before[warp] = before, s_all[warp] = all;
    __syncthreads();
    before = all = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) before += s_before[w], all += s_all[w];
    walk.look(a, tile.seq, kRows, false);
    const int64_t ctas = a.partial_bytes / (2 * kRows * (D + 2) * 4), per = (all + ctas - 1) / ctas;
    before += ((int64_t)(tile.r0 / kRows) * a.c.heads + h) * walk.weight;
    const int64_t from = (before + kOpening) / per, n = per * (from + 1) - before;   // the CTA that begins it, and as much of it
    const int first = (int)from, pieces = n >= walk.weight ? 1 : 1 + (int)((walk.weight - n + per - 1) / per);
    grid_dependency_wait();   // launched while the parts are still being made
    if (pieces <= 1 || pieces > ctas - first) return;
    [[maybe_unused]] const int64_t o_bytes =
        ((a.b.rows - 1) * a.O.row + (a.q_heads - 1) * a.O.head + D) * (int64_t)sizeof(T);
    const int member = warp % TEAM, r = blockIdx.z * (8 / TEAM) + warp / TEAM;
    if (TEAM == 1 ? tile.r0 + r >= tile.nrows : tile.r0 + (int)blockIdx.z >= tile.nrows) return;   // of a team all or none
    auto part = [&](int i) { return a.partial + ((int64_t)(first + i) * 2 + (i == 0 ? 1 : 0)) * (kRows * (D + 2)); };
    const int share = (pieces + TEAM - 1) / TEAM, end = min(pieces, (member + 1) * share);
    float top = kLowest, sum = 0.0f, acc[kEach] = {};
    float m[kBatch], l[kBatch], x[kBatch][kEach];
    auto load = [&](int i0) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            m[b] = kLowest, l[b] = 0.0f;
#pragma unroll
            for (int e = 0; e < kEach; ++e) x[b][e] = 0.0f;
            if (i0 + b >= end) continue;
            const float *at = part(i0 + b), *ml = at + kRows * D + 2 * r;
            if (!GEMM_DBG_OK(ml, a.partial, a.partial_bytes, 8)) continue;
            m[b] = ml[0], l[b] = ml[1];
#pragma unroll
            for (int e = 0; e < kEach; ++e) x[b][e] = at[r * D + lane + 32 * e];
        }
    };
    load(member * share);   // under way together with the maxima
    for (int i = lane; i < pieces; i += 32) {
        const float* ml = part(i) + kRows * D + 2 * r;
        if (GEMM_DBG_OK(ml, a.partial, a.partial_bytes, 8)) top = fmaxf(top, ml[0]);
    }
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, i));
    for (int i = member * share; i < end; i += kBatch) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (i + b >= end) break;
            const float f = exp2_approx(m[b] - top);
            sum = fmaf(f, l[b], sum);
#pragma unroll
            for (int e = 0; e < kEach; ++e) acc[e] = fmaf(f, x[b][e], acc[e]);
        }
        if (i + kBatch < end) load(i + kBatch);
    }
    if constexpr (TEAM > 1) {
#pragma unroll
        for (int e = 0; e < kEach; ++e) s_acc[member][lane + 32 * e] = acc[e];
        if (lane == 0) s_sum[member] = sum;
        __syncthreads();
        if (member > 0) return;
#pragma unroll
        for (int w = 1; w < TEAM; ++w) {
            sum += s_sum[w];
#pragma unroll
            for (int e = 0; e < kEach; ++e) acc[e] += s_acc[w][lane + 32 * e];
        }
    }
    T* dst = out_row<T>(a, tile, h, tile.r0 + r) + lane;
#pragma unroll
    for (int e = 0; e < kEach; ++e)
        if (GEMM_DBG_OK(dst + 32 * e, a.O.p, o_bytes, sizeof(T))) dst[32 * e] = from_float<T>(sum == 0.0f ? 0.0f : acc[e] / sum);
}

template <typename T, int D, int NQ>
cudaError_t launch(const AttnArgs& a, const KvPlan& plan, int* launches, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Ring<D, NQ>::kBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    *launches = 1;
    if (plan.ctas == 0) {
        cfg.gridDim = dim3((unsigned)(plan.units * plan.splits), (unsigned)a.c.heads);
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = (unsigned)plan.splits;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        return cudaLaunchKernelEx(&cfg, kv4_cluster_kernel<T, D, NQ>, a);
    }
    cfg.gridDim = dim3((unsigned)plan.ctas);
    cfg.numAttrs = 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kv4_line_kernel<T, D, NQ>, a);
    if (e != cudaSuccess) return e;
    *launches = 2;
    // 8 heads over 32768 and 200000 tokens: 18.7 and 48.4 us with a team of warps a
    // row, 23.2 and 53.5 with one warp; 64 sequences of up to 8192: 84 and 67.
    const bool team = plan.ctas > 8 * plan.units * a.c.heads;
    cfg.gridDim = dim3((unsigned)plan.units, (unsigned)a.c.heads, team ? plan.rows : NQ);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = kUsePdl;
    cfg.numAttrs = 1;
    return team ? cudaLaunchKernelEx(&cfg, kv4_line_join_kernel<T, D, NQ, 8>, a) : cudaLaunchKernelEx(&cfg, kv4_line_join_kernel<T, D, NQ, 1>, a);
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
                    using T = decltype(t);
                    constexpr int D = decltype(d)::value, NQ = decltype(nq)::value;
                    const auto most = cudaFuncAttributeMaxDynamicSharedMemorySize;
                    const cudaError_t c = cudaFuncSetAttribute(kv4_cluster_kernel<T, D, NQ>, most, Ring<D, NQ>::kBytes);
                    return c != cudaSuccess ? c : cudaFuncSetAttribute(kv4_line_kernel<T, D, NQ>, most, Ring<D, NQ>::kBytes);
                });
                if (e != cudaSuccess) return e;
            }
    return cudaSuccess;
}

cudaError_t launch_kv4_few(const AttnArgs& a, ElemType type, const KvPlan& plan, int* launches, cudaStream_t stream) {
    return with_kernel(type, a.c.dim, plan.rows, [&](auto t, auto d, auto nq) {
        return launch<decltype(t), decltype(d)::value, decltype(nq)::value>(a, plan, launches, stream);
    });
}

// The host's part of launch_kv4_few: how few rows' tokens are shared.  A cluster a
// tile is one launch, and no CTA has to find its piece: 8 heads over up to 1000
// tokens take 6.7 us for one sequence (in a line 8.9) and 8.4 for 6 (11.5), over up
// to 8192 tokens 12.3 for one (12.0) and 16.7 for 6 (17.2).  But clusters of eight do
// not find the last of the GPU's slots: with 448 CTAs for 456 slots, 7 sequences,
// 1000 tokens take 13.2 us (11.6), hence seven eighths.
void kv4_few_plan(KvPlan& p, const KvView& c, int64_t have, int64_t most, int num_sms) {
    const int64_t slots = (int64_t)resident(p.rows / 8) * num_sms;
    p.ctas = 0;
    p.cluster = true;
    p.scratch_bytes = 0;
    if (most <= 8 * kMaxCluster && 8 * have * (most < kMaxCluster ? most : kMaxCluster) <= 7 * slots) {
        p.splits = (int)(most < 1 ? 1 : most < kMaxCluster ? most : kMaxCluster);
        return;
    }
    p.splits = 1;
    const int64_t line = have * (most + kOpening);
    p.ctas = (int)(line < slots ? line : slots);
    p.scratch_bytes = (int64_t)p.ctas * 2 * (p.rows * (c.dim + 2) * 4);
}

}  // namespace libgemm
