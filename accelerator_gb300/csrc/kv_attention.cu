// kv_attention.cu -- attention of ragged queries over the paged 8-bit cache.
//
// For each query row  o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale * q.k_j
// - m), in one pass over the tokens with the running maximum m and sum; keys
// and values are code * scale of their page, so the page's key scale goes
// onto the score and its value scale onto p_j, and the codes themselves enter
// both products exactly, as binary16 integers.  The query heads that share a
// cache head, and the queries of a sequence, are the rows of one tile.
#include "kv_attention.cuh"

namespace libgemm {
namespace {

constexpr int kWarps = 4;        // warps that compute; one more copies
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kSub = 16;         // tokens of one product, all of one page
constexpr int kSubs = 2;         // a warp takes this many times 16 tokens at once
constexpr int kStep = kWarps * kSubs * kSub;   // tokens of a stage
constexpr int kRingBytes = 96 * 1024;  // two CTAs of an SM keep 192 KB in flight
constexpr int kMaxCluster = 8;
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

// What the copying warp tells the others about 16 tokens of a stage.
struct SubInfo {
    float ks, vs;
    uint32_t live;
    uint32_t pad;
};

template <int D>
struct Ring {
    static constexpr int kStageBytes = 2 * kStep * D;
    static constexpr int kStages = kRingBytes / kStageBytes;   // 3 for 128, 6 for 64
    // [stages][keys, values][128][D], then SubInfo[stages][8], then the barriers
    static constexpr int kInfoAt = kStages * kStageBytes;
    static constexpr int kBarsAt = kInfoAt + kStages * kWarps * kSubs * (int)sizeof(SubInfo);
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

// Few query rows: a tile of 8 * NQ rows over a share of its tokens.  One warp
// copies whole pages' parts into a ring of stages of 128 tokens (their codes
// lie in one piece for a page and head), four take 32 tokens of each stage.
// Both products have the tokens' side, of which there is much, as the 16-row
// operand and the queries as its eight columns: S^T = K Q^T, then O^T = V^T
// P^T, for which the weights are turned over in registers; a product of 16
// query rows would be half empty for the usual eight or fewer heads to a key
// head (in that form the example below took 250 us, in this one 160, all else
// as it then was).
//
// Bound by reading the codes while a CTA is under way: 64 sequences of up to
// 8192 tokens, 64 heads over 8 of 128, 613 MB in 125 us, 4.9 TB/s or 72 % of the
// measured copy rate, and 6 TB/s between a CTA's first stage and its last.  The
// rest is its beginning (3 us until its copies are under way) and its end (4 us
// to join), which the SM's other CTA covers in part; more, smaller shares of a
// sequence only add to them (2 shares 130 us, 4 155, 8 218 when it was chosen).
template <typename T, int D, int NQ>
__global__ void __launch_bounds__(kThreads, 2) kv_attention_kernel(const AttnArgs a) {
    using R = Ring<D>;
    constexpr int kRows = 8 * NQ, kLd = D + 4;
    static_assert(kWarps * kRows * (kLd + 2) * 4 + 8 * kRows <= R::kInfoAt, "the joining reuses the ring");
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t ring = smem_u32(smem), bars = ring + R::kBarsAt;   // full[stages], empty[stages]
    SubInfo* info = reinterpret_cast<SubInfo*>(smem + R::kInfoAt);
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
        const int log2 = a.c.page_log2, chunk = min(kStep, 1 << log2);   // tokens of one copy
        [[maybe_unused]] const int64_t code_bytes = a.c.pages * a.c.heads * ((int64_t)D << log2);
        SubInfo mine = {};
        int64_t from = 0;
        uint32_t phase = 0;
        int stage = 0, issued = 0;
        for (int s = 0; s < steps; ++s) {
            if (s % 4 == 0) {
                const int tok = tok_begin + s * kStep + lane * kSub;
                bool live = tile.page_seen(tok, log2);
                const int64_t page = live ? __ldg(table + (tok >> log2)) : 0;
                if (live && (page < 0 || page >= a.c.pages)) {
                    atomicOr(a.err, kErrIndex);
                    live = false;
                }
                const int64_t ph = page * a.c.heads + h;
                mine.live = live;
                mine.ks = live ? __ldg(a.c.ks + ph) : 0.0f;
                mine.vs = live ? __ldg(a.c.vs + ph) : 0.0f;
                from = ((ph << log2) + (tok & ((1 << log2) - 1))) * D;
            }
            if (!warp_wait(bars + 8 * (R::kStages + stage), phase ^ 1u, abort_flag, a.err)) break;
            const int sub = lane - s % 4 * 8;   // this lane's part of the stage, if it has one
            const bool here = sub >= 0 && sub < 8;
            // the first 16 tokens of a page's part fetch all of it
            bool copies = here && mine.live && sub * kSub % chunk == 0;
            if (copies) copies = GEMM_DBG_OK(a.c.k + from, a.c.k, code_bytes, chunk * D) && GEMM_DBG_OK(a.c.v + from, a.c.v, code_bytes, chunk * D);
            const int parts = __popc(__ballot_sync(0xFFFFFFFFu, copies));
            // The copies go first, then the scales, which may still be on their
            // way; the stage is not full before the arrival below.
            if (copies) {
                const uint32_t to = ring + stage * R::kStageBytes + sub * kSub * D;
                bulk_load(to, a.c.k + from, chunk * D, bars + 8 * stage);
                bulk_load(to + kStep * D, a.c.v + from, chunk * D, bars + 8 * stage);
            }
            if (here) info[stage * 8 + sub] = mine;
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(bars + 8 * stage, (uint32_t)(parts * 2 * chunk * D));
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
        // Query row 8n + g as the column g of B.  A lane's part of a row is 16
        // neighbours of each 64: its k of four instructions, in the order in
        // which its 16 bytes of a key row hold them.  bfloat16 rows are brought
        // to [1, 2) by a power of two (exact, but for elements under 2^-14 of the
        // row's largest, whose error stays under 2^-25 of it) to be binary16.
        uint32_t qf[NQ][D / 16][2];
        float row_scale[NQ][2];      // of the rows 8n + 2t, + 1, whose scores a lane gets
        int row_lo[NQ][2], row_hi[NQ][2];
        [[maybe_unused]] const int64_t q_bytes =
            ((a.b.rows - 1) * a.Q.row + (a.q_heads - 1) * a.Q.head + D) * (int64_t)sizeof(T);
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const unsigned r = tile.r0 + 8 * n + g;
            const bool live = r < (unsigned)tile.nrows;
            const T* p = static_cast<const T*>(a.Q.p) + (int64_t)(tile.row0 + (live ? r / a.share : 0)) * a.Q.row +
                         (int64_t)(h * a.share + (live ? r % a.share : 0)) * a.Q.head;
            Eight<T> x[D / 64][2] = {};
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const T* pe = p + 64 * j + 16 * t + 8 * e;
                    if (live && GEMM_DBG_OK(pe, a.Q.p, q_bytes, 16)) x[j][e] = load_eight(pe, a.q_vec);
                }
            float up = 1.0f, down = 1.0f;
            if constexpr (!std::is_same<T, __half>::value) {
                float top = 0.0f;
#pragma unroll
                for (int j = 0; j < D / 64; ++j)
#pragma unroll
                    for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(x[j][e / 8].at(e % 8)));
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                const int e = (int)(__float_as_uint(top) >> 23);   // biased exponent
                if (top > 0.0f && top < INFINITY) {
                    const int k = max(1, min(253, e));
                    up = __uint_as_float((uint32_t)k << 23);             // 2^(k - 127)
                    down = __uint_as_float((uint32_t)(254 - k) << 23);   // 2^(127 - k)
                }
            }
            if (a.scale_log2 < 0.0f) down = -down;   // the scores' scale is positive from here on
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const Eight<T>& e = x[j][s / 2];
                    const int o = 4 * (s % 2);
                    qf[n][4 * j + s][0] = pack2<__half>(e.at(o) * down, e.at(o + 1) * down);
                    qf[n][4 * j + s][1] = pack2<__half>(e.at(o + 2) * down, e.at(o + 3) * down);
                }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                row_scale[n][i] = fabsf(a.scale_log2) * __shfl_sync(0xFFFFFFFFu, up, 4 * (2 * t + i));
                // rows past the last one see all: they are not stored
                const int rr = tile.r0 + 8 * n + 2 * t + i;
                row_lo[n][i] = rr < tile.nrows ? tile.row_lo(a, rr) : 0;
                row_hi[n][i] = rr < tile.nrows ? tile.row_hi(a, rr) : tile.hi;
            }
        }
        // tokens that every row of the tile sees
        const int full_lo = tile.row_lo(a, min(tile.r0 + kRows, tile.nrows) - 1);
        const int full_hi = tile.row_hi(a, tile.r0);

        constexpr int MT = D / 16;      // row tiles of O^T: row g of tile i is d = g * D / 8 + 2i, row g + 8 the next
        // A row's sums: l of the weights exp2(s_j - m) in binary32, o of those times
        // their page's value scale v_j times up = 2^15 / r as binary16, where m and r
        // are the row's own largest s_j and exp2(s_j - m) * v_j so far, of tokens that
        // it sees (r at least kLeast, so that up stays finite).
        float o[NQ][MT][4], m[NQ][2], l[NQ][2], up[NQ][2];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
#pragma unroll
            for (int i = 0; i < MT; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.0f;
            m[n][0] = m[n][1] = kLowest;
            l[n][0] = l[n][1] = 0.0f;
            up[n][0] = up[n][1] = kPScale / kLeast;
        }

        uint32_t phase = 0;
        int stage = 0;
        for (int s = 0; s < steps; ++s) {
            if (!warp_wait(bars + 8 * stage, phase, abort_flag, a.err)) break;
            const SubInfo* in = info + (stage * kWarps + warp) * kSubs;
            const uint32_t kat = ring + stage * R::kStageBytes + warp * (kSubs * kSub * D), vat = kat + kStep * D;
            const int tok = tok_begin + s * kStep + warp * (kSubs * kSub);
            if (tok < tile.hi) {
                // scores of tokens 16b + g and 16b + g + 8 for the rows 2t, 2t + 1
                float sc[kSubs][NQ][4], f[kSubs][NQ][2];
#pragma unroll
                for (int b = 0; b < kSubs; ++b) {
                    float part[NQ][2][4] = {};
#pragma unroll
                    for (int j = 0; j < D / 64; ++j) {
                        const uint32_t at = kat + (16 * b + g) * D + 64 * j + 16 * t;
                        const uint4 w0 = lds128(at), w1 = lds128(at + 8 * D);
                        const uint32_t lo[4] = {w0.x, w0.y, w0.z, w0.w}, hi[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t a0 = codes01(lo[k]), a1 = codes01(hi[k]), a2 = codes23(lo[k]), a3 = codes23(hi[k]);
#pragma unroll
                            for (int n = 0; n < NQ; ++n)
                                mma_16816<__half>(part[n][k & 1], a0, a1, a2, a3, qf[n][4 * j + k][0], qf[n][4 * j + k][1]);
                        }
                    }
                    const float ks = in[b].ks;
#pragma unroll
                    for (int n = 0; n < NQ; ++n) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) sc[b][n][e] = part[n][0][e] + part[n][1][e];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            // a page of zeros has scale 0: above 0, so that a hidden token's -inf stays that
                            f[b][n][i] = row_scale[n][i] * ks;
                            if (f[b][n][i] < 1.1754943508222875e-38f) f[b][n][i] = 1.1754943508222875e-38f;
                        }
                    }
                    // Tokens that some row does not see, pages that do not exist.
                    const bool live = in[b].live != 0;
                    if (tok + 16 * b < full_lo || tok + 16 * b + kSub > full_hi || !live) {
#pragma unroll
                        for (int n = 0; n < NQ; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int j = tok + 16 * b + g + 8 * (e >> 1);
                                if (j < row_lo[n][e & 1] || j >= row_hi[n][e & 1] || !live) sc[b][n][e] = kNegInf;
                            }
                        asm volatile("");   // a branch: few tokens come here
                    }
                    if (ks != ks) {   // a page that reads as NaN: for the rows that see it alone
#pragma unroll
                        for (int n = 0; n < NQ; ++n) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) sc[b][n][e] = sc[b][n][e] == kNegInf ? kNegInf : ks;
                            f[b][n][0] = f[b][n][1] = 1.0f;
                        }
                    }
                }
                const float vs[2] = {in[0].vs, in[1].vs};
                // A page's value scale for a row: finite, so that a weight of 0 stays 0;
                // where it is held to 2^127 the weights are under 2^-111.
                auto factor = [&](int b, int n, int i) { return fminf(vs[b] * up[n][i], 1.7014118e38f); };
                float w[kSubs][NQ][4];
                auto weigh = [&] {   // returns the largest weight of either product
                    float most = 0.0f;
#pragma unroll
                    for (int b = 0; b < kSubs; ++b)
#pragma unroll
                        for (int n = 0; n < NQ; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                w[b][n][e] = exp2_approx(fmaf(sc[b][n][e], f[b][n][e & 1], -m[n][e & 1]));
                                most = max3(most, w[b][n][e], w[b][n][e] * factor(b, n, e & 1));
                            }
                    return most;
                };
                // The sums so far are brought to new maxima only when one is passed
                // by so much that a weight might not fit binary16.
                if (__any_sync(0xFFFFFFFFu, weigh() > kMostP)) {
#pragma unroll
                    for (int n = 0; n < NQ; ++n) {
                        float grow[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float t0 = fmaxf(sc[0][n][i], sc[0][n][2 + i]) * f[0][n][i];
                            const float t1 = fmaxf(sc[1][n][i], sc[1][n][2 + i]) * f[1][n][i];
                            float top = fmaxf(t0, t1);
                            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 4));
                            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 8));
                            top = fmaxf(fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16)), m[n][i]);
                            const float keep = exp2_approx(m[n][i] - top), held = keep * __fdividef(kPScale, up[n][i]);
                            m[n][i] = top;
                            l[n][i] *= keep;
                            float rel = fmaxf(exp2_approx(t0 - top) * vs[0], exp2_approx(t1 - top) * vs[1]);
                            rel = fmaxf(rel, __shfl_xor_sync(0xFFFFFFFFu, rel, 4));
                            rel = fmaxf(rel, __shfl_xor_sync(0xFFFFFFFFu, rel, 8));
                            rel = fmaxf(rel, __shfl_xor_sync(0xFFFFFFFFu, rel, 16));
                            rel = max3(rel, held, kLeast);
                            up[n][i] = __fdividef(kPScale, rel);
                            grow[i] = __fdividef(held, rel);   // 1 at most
                        }
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            o[n][i][0] *= grow[0], o[n][i][1] *= grow[1];
                            o[n][i][2] *= grow[0], o[n][i][3] *= grow[1];
                        }
                    }
                    weigh();
                }
#pragma unroll
                for (int b = 0; b < kSubs; ++b) {
                    uint32_t vw[4][D / 32];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t at = vat + (16 * b + 8 * (i >> 1) + 2 * t + (i & 1)) * D + g * (D / 8);
                        if constexpr (D == 128) {
                            const uint4 x = lds128(at);
                            vw[i][0] = x.x, vw[i][1] = x.y, vw[i][2] = x.z, vw[i][3] = x.w;
                        } else {
                            const uint2 x = lds64(at);
                            vw[i][0] = x.x, vw[i][1] = x.y;
                        }
                    }
                    // Binary16 under 2^16, normal down to 2^-29 of the row's largest.
                    uint32_t pt[NQ][2];
#pragma unroll
                    for (int n = 0; n < NQ; ++n) {
                        float p[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) p[e] = w[b][n][e] * factor(b, n, e & 1);
                        if (vs[b] != vs[b]) {   // a page that reads as NaN, likewise
#pragma unroll
                            for (int e = 0; e < 4; ++e) p[e] = sc[b][n][e] == kNegInf ? 0.0f : vs[b];
                        }
                        l[n][0] += w[b][n][0] + w[b][n][2];
                        l[n][1] += w[b][n][1] + w[b][n][3];
                        pt[n][0] = transpose8(pack2<__half>(p[0], p[1]));
                        pt[n][1] = transpose8(pack2<__half>(p[2], p[3]));
                    }
#pragma unroll
                    for (int e = 0; e < D / 32; ++e) {
                        const uint32_t a01 = __byte_perm(vw[0][e], vw[1][e], 0x5140), a23 = __byte_perm(vw[0][e], vw[1][e], 0x7362);
                        const uint32_t b01 = __byte_perm(vw[2][e], vw[3][e], 0x5140), b23 = __byte_perm(vw[2][e], vw[3][e], 0x7362);
                        const uint32_t f0[4] = {codes01(a01), codes23(a01), codes01(b01), codes23(b01)};
                        const uint32_t f1[4] = {codes01(a23), codes23(a23), codes01(b23), codes23(b23)};
#pragma unroll
                        for (int n = 0; n < NQ; ++n) {
                            mma_16816<__half>(o[n][2 * e], f0[0], f0[1], f0[2], f0[3], pt[n][0], pt[n][1]);
                            mma_16816<__half>(o[n][2 * e + 1], f1[0], f1[1], f1[2], f1[3], pt[n][0], pt[n][1]);
                        }
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
                const float unit = 1.0f / up[n][i];
                l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], 4);
                l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], 8);
                l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], 16);
                if (g == 0) s_m[at] = m[n][i], s_l[at] = l[n][i];
                float4* row = reinterpret_cast<float4*>(s_o + at * kLd + g * (D / 8));
#pragma unroll
                for (int e = 0; e < MT / 2; ++e)
                    row[e] = make_float4(o[n][2 * e][i] * unit, o[n][2 * e][2 + i] * unit, o[n][2 * e + 1][i] * unit,
                                         o[n][2 * e + 1][2 + i] * unit);
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

// Joins the splits of a tile's rows, in order.  GROUPS teams of LANES threads
// share a row's splits: a block of 1024 to a row where rows are few and splits
// many, so that all loads are in flight at once, a warp to a row where it is
// the other way.
template <typename T, int D, int LANES, int GROUPS, int THREADS>
__global__ void __launch_bounds__(THREADS) kv_join_kernel(const AttnArgs a, int rows, int step) {
    constexpr int kEach = D / LANES, kAtOnce = THREADS / (LANES * GROUPS);   // elements of a thread, rows of a block
    __shared__ float s_acc[GROUPS][kAtOnce][D], s_sum[GROUPS][kAtOnce];
    const int u = blockIdx.x, h = blockIdx.y;
    const int lane = threadIdx.x % LANES, q = threadIdx.x / LANES % GROUPS, mine = threadIdx.x / (LANES * GROUPS);
    Tile tile;
    const bool found = tile.find(a, u, rows, step, false);
    grid_dependency_wait();   // launched while the partial results are still being made
    if (!found || tile.active == 1) return;
    const int64_t slot = (int64_t)rows * (D + 2);
    const float* part = a.partial + ((int64_t)u * a.c.heads + h) * a.splits * slot;
    const int share = (tile.active + GROUPS - 1) / GROUPS, end = min(tile.active, (q + 1) * share);
    const int r = blockIdx.z * kAtOnce + mine;
    const bool live = tile.r0 + r < tile.nrows;
    float sum = 0.0f, acc[kEach] = {};
    if (live) {
        const float* ml = part + rows * D + 2 * r;
        float top = kLowest;
        for (int s = threadIdx.x % 32; s < tile.active; s += 32)
            if (GEMM_DBG_OK(ml + s * slot, a.partial, a.partial_bytes, 8)) top = fmaxf(top, ml[s * slot]);
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, i));   // a warp has one row
#pragma unroll 8
        for (int s = q * share; s < end; ++s) {
            const float f = exp2_approx(ml[s * slot] - top);
            sum = fmaf(f, ml[s * slot + 1], sum);
#pragma unroll
            for (int e = 0; e < kEach; ++e) acc[e] = fmaf(f, part[s * slot + r * D + lane + e * LANES], acc[e]);
        }
    }
    if constexpr (GROUPS > 1) {
        if (live) {
#pragma unroll
            for (int e = 0; e < kEach; ++e) s_acc[q][mine][lane + e * LANES] = acc[e];
            if (lane == 0) s_sum[q][mine] = sum;
        }
        __syncthreads();
        if (q != 0) return;
        if (live) {
#pragma unroll
            for (int g = 1; g < GROUPS; ++g) {
                sum += s_sum[g][mine];
#pragma unroll
                for (int e = 0; e < kEach; ++e) acc[e] += s_acc[g][mine][lane + e * LANES];
            }
        }
    }
    if (!live) return;
    [[maybe_unused]] const int64_t o_bytes =
        ((a.b.rows - 1) * a.O.row + (a.q_heads - 1) * a.O.head + D) * (int64_t)sizeof(T);
    T* dst = out_row<T>(a, tile, h, tile.r0 + r) + lane;
#pragma unroll
    for (int e = 0; e < kEach; ++e)
        if (GEMM_DBG_OK(dst + e * LANES, a.O.p, o_bytes, sizeof(T))) dst[e * LANES] = from_float<T>(sum == 0.0f ? 0.0f : acc[e] / sum);
}

template <typename T, int D, int NQ>
cudaError_t launch(const AttnArgs& a, const KvPlan& plan, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(plan.units * plan.splits), (unsigned)a.c.heads);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Ring<D>::kBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = a.partial ? 1 : (unsigned)plan.splits;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_attention_kernel<T, D, NQ>, a);
}

template <typename T, int D>
cudaError_t launch(const AttnArgs& a, const KvPlan& plan, int* launches, cudaStream_t stream) {
    const ElemType type = std::is_same<T, __half>::value ? ElemType::kF16 : ElemType::kBF16;
    cudaError_t e = plan.rows == 8    ? launch<T, D, 1>(a, plan, stream)
                    : plan.rows == 16 ? launch<T, D, 2>(a, plan, stream)
                                      : launch_kv_prompt(a, type, plan, stream);
    *launches = 1;
    if (e == cudaSuccess && a.partial) {
        static_assert(kStep == 128, "both kernels count tokens in the same steps");
        cudaLaunchConfig_t cfg = {};
        const bool many = plan.rows == 256;
        cfg.gridDim = dim3((unsigned)plan.units, (unsigned)a.c.heads, (unsigned)(many ? plan.rows / 8 : plan.rows));
        cfg.blockDim = dim3(many ? 256 : 1024);
        cfg.stream = stream;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = kUsePdl;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        e = many ? cudaLaunchKernelEx(&cfg, kv_join_kernel<T, D, 32, 1, 256>, a, plan.rows, kStep)
                 : cudaLaunchKernelEx(&cfg, kv_join_kernel<T, D, D, 1024 / D, 1024>, a, plan.rows, kStep);
        *launches = 2;
    }
    return e;
}

template <typename T, int D>
cudaError_t allow_smem() {
    const cudaError_t e = cudaFuncSetAttribute(kv_attention_kernel<T, D, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               Ring<D>::kBytes);
    return e != cudaSuccess ? e
                            : cudaFuncSetAttribute(kv_attention_kernel<T, D, 2>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, Ring<D>::kBytes);
}

}  // namespace

LIBGEMM_DEBUG_READER(kv_attention_debug_flags)

cudaError_t kv_attention_setup() {
    cudaError_t e = allow_smem<__nv_bfloat16, 64>();
    if (e == cudaSuccess) e = allow_smem<__nv_bfloat16, 128>();
    if (e == cudaSuccess) e = allow_smem<__half, 64>();
    if (e == cudaSuccess) e = allow_smem<__half, 128>();
    return e == cudaSuccess ? kv_prompt_setup() : e;
}

// How many rows a tile has follows from the rows of a sequence and cache head,
// on average: up to 8 and up to kPromptRows the kernel for few rows, in tiles of
// 8 and 16, beyond that the one on the tensor memory, although its 128-row
// products are then three quarters empty: a tile of 16 reads all of the cache
// again.  4 sequences over 4000 tokens of 8 heads of 128, two query heads to each:
// of 31 queries 77 us in tiles of 16 and 49 in one of 256, of 17 queries 63 and
// 47, of 16 queries 46 in two tiles of 16.  (With 2 cache heads, too few tiles to
// fill the GPU, 17 and 31 queries take 28 us in tiles of 16 and 38 in one of 256,
// and batches that mix prompts and single tokens take one kernel for both.)
//
// Few rows: tiles that fill an eighth of the GPU's CTA slots or more, or whose
// tokens are few, have their tokens shared over a cluster (joined through
// distributed shared memory, no second launch), two rounds of CTAs in all, as
// sequences differ in length.  Fewer tiles over long sequences are shared over
// one round of CTAs and joined by a second kernel.  Many rows: the tokens are
// shared, and joined likewise, only if the tiles leave half the GPU idle.
constexpr int64_t kPromptRows = 32;

int64_t gcd(int64_t a, int64_t b) { return b ? gcd(b, a % b) : a; }

KvPlan kv_plan(const KvView& c, const KvBatch& b, int q_heads, int64_t window, int num_sms) {
    KvPlan p;
    const int64_t share = q_heads / c.heads, all = b.rows * share;
    p.rows = all <= 8 * (int64_t)b.sequences    ? 8
             : all <= kPromptRows * b.sequences ? 16
                                                : 256;
    const int64_t tiles = all / p.rows;
    p.gap = p.rows - (int)gcd(p.rows, share);
    p.units = (all + b.sequences * (int64_t)p.gap) / p.rows;   // at least the tiles that there are
    int64_t longest = b.width << c.page_log2;
    if (window > 0 && window < longest - p.rows - 2 * kStep) longest = window + p.rows + 2 * kStep;
    if (p.units < 1) p.units = 1;
    const int64_t have = (tiles > b.sequences ? tiles : b.sequences) * c.heads, slots = (p.rows == 256 ? 1 : 2) * (int64_t)num_sms;
    const int64_t most = (longest + kStep - 1) / kStep;
    int64_t splits;
    if (p.rows == 256) {
        splits = slots / have;
        if (splits > most / 4) splits = most / 4;
        p.cluster = false;
    } else {
        p.cluster = most <= 8 * kMaxCluster || have * kMaxCluster >= slots;
        splits = p.cluster ? (2 * slots + have - 1) / have : slots / have;
        if (splits > most) splits = most;
        if (p.cluster && splits > kMaxCluster) splits = kMaxCluster;
    }
    p.splits = (int)(splits < 1 ? 1 : splits);
    p.scratch_bytes = p.splits > 1 && !p.cluster ? p.units * c.heads * p.splits * (p.rows * (c.dim + 2) * 4) : 0;
    return p;
}

cudaError_t launch_kv_attention(const KvView& c, const KvRows& Q, const KvRows& O, ElemType type,
                                int q_heads, float scale, bool causal, int64_t window,
                                const KvBatch& b, const KvPlan& plan, void* scratch,
                                unsigned* err, int* launches, cudaStream_t stream) {
    const bool q_vec = (reinterpret_cast<uintptr_t>(Q.p) & 15u) == 0 && Q.row % 8 == 0 && Q.head % 8 == 0;
    const AttnArgs a{c, Q, O, b, q_heads, (unsigned)(q_heads / c.heads), plan.gap, scale * 1.44269504088896341f, causal,
                     (int)(window < INT32_MAX ? window : INT32_MAX), plan.splits, q_vec, plan.scratch_bytes, static_cast<float*>(scratch), err};
    if (type == ElemType::kBF16)
        return c.dim == 128 ? launch<__nv_bfloat16, 128>(a, plan, launches, stream)
                            : launch<__nv_bfloat16, 64>(a, plan, launches, stream);
    return c.dim == 128 ? launch<__half, 128>(a, plan, launches, stream)
                        : launch<__half, 64>(a, plan, launches, stream);
}

}  // namespace libgemm
