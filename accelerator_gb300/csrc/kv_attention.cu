// kv_attention.cu -- attention of ragged queries over the paged 8-bit cache.
//
// For each query row  o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale * q.k_j
// - m), in one pass over the tokens with the running maximum m and sum; keys
// and values are code * scale of their page, so the page's key scale goes
// onto the score and its value scale onto p_j, and the codes themselves enter
// both products exactly, as binary16 integers.  The query heads that share a
// cache head, and the queries of a sequence, are the rows of one tile.
#include <type_traits>

#include "kernels.h"
#include "lowbit.cuh"

namespace libgemm {
namespace {

constexpr int kRows = 16;        // query rows of a tile (one m16 matrix instruction)
constexpr int kWarps = 4;        // warps that compute; one more copies
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kSub = 16;         // tokens a warp takes at once
constexpr int kStep = kWarps * kSub;   // tokens of a stage
constexpr int kMinSteps = 2;     // stages of a split, at least
constexpr int kRingBytes = 96 * 1024;  // two CTAs of an SM keep 192 KB in flight
constexpr int kMaxCluster = 8;
constexpr float kNegInf = -INFINITY;
constexpr float kPScale = 32768.0f;   // weights enter the second product times 2^15
constexpr uint64_t kWaitLimitNs = 2000000000ull;

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

struct AttnArgs {
    KvView c;
    KvRows Q, O;
    KvBatch b;
    int q_heads, share;          // query heads, and how many read one cache head
    float scale_log2;            // scale * log2(e)
    int causal;
    int64_t window;
    int splits;                  // CTAs that share a tile's tokens: a cluster, or with `partial` any number
    bool q_vec;                  // Q in 16-byte loads
    float* partial;              // [unit][head][split] x (kRows x dim sums, then kRows x (max, sum))
    unsigned* err;
};

// The tile of a unit: its sequence and rows, and the tokens that it sees.
struct Tile {
    int seq;
    int64_t row0;                // first of the sequence's rows
    int64_t r0, nrows;           // first row (query, head pair) of the tile; rows of the sequence
    int64_t len, p0;             // cached tokens; position of query 0
    int64_t tok0;                // first token, a multiple of kStep
    int64_t hi;                  // end of the tokens any row sees
    int steps, per, active;      // steps in all, per split, splits that have any

    __device__ __forceinline__ int64_t row_hi(const AttnArgs& a, int64_t r) const {
        if (r >= nrows) return 0;
        const int64_t p = p0 + r / a.share;
        if (p < 0) return 0;
        return a.causal ? p + 1 : len;
    }
    __device__ __forceinline__ int64_t row_lo(const AttnArgs& a, int64_t r) const {
        const int64_t p = p0 + r / a.share;
        return a.window > 0 && p >= a.window ? p - a.window + 1 : 0;
    }
    __device__ __forceinline__ bool find(const AttnArgs& a, int64_t u, bool report) {
        const Starts starts{a.b.starts, a.b.sequences, a.b.rows};
        // Sequence q's tiles are units floor(starts[q] * share / 16) + q + j.
        seq = last_not_above(a.b.sequences, u, [&](int i) { return starts.at(i) * a.share / kRows + i; });
        row0 = starts.at(seq);
        const int64_t count = starts.at(seq + 1) - row0;
        if (!starts.whole(u == 0, seq)) {
            if (report) atomicOr(a.err, kErrIndex);
            return false;
        }
        nrows = count * a.share;
        r0 = (u - row0 * a.share / kRows - seq) * kRows;
        if (r0 < 0 || r0 >= nrows) return false;
        len = __ldg(a.b.at + seq);
        if (len < 0 || len > (a.b.width << a.c.page_log2)) {
            if (report) atomicOr(a.err, kErrIndex);
            len = 0;
        }
        p0 = len - count;
        const int64_t last = r0 + kRows - 1 < nrows ? r0 + kRows - 1 : nrows - 1;
        hi = row_hi(a, last);
        tok0 = row_lo(a, r0) / kStep * kStep;
        steps = hi > tok0 ? (int)((hi - tok0 + kStep - 1) / kStep) : 0;
        per = (steps + a.splits - 1) / a.splits;
        if (per < kMinSteps) per = kMinSteps;
        active = (steps + per - 1) / per;
        if (active < 1) active = 1;
        return true;
    }
};

// Where a row's results go.
template <typename T>
__device__ __forceinline__ T* out_row(const AttnArgs& a, const Tile& tile, int h, int64_t r) {
    return static_cast<T*>(a.O.p) + (tile.row0 + r / a.share) * a.O.row + (h * a.share + r % a.share) * a.O.head;
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

// What the copying warp tells the others about 16 tokens of a stage.
struct SubInfo {
    float ks, vs;
    uint32_t live;
    uint32_t pad;
};

template <int D>
struct Ring {
    static constexpr int kStageBytes = 2 * kStep * D;
    static constexpr int kStages = kRingBytes / kStageBytes;   // 6 for 128, 12 for 64
    // [stages][keys, values][64][D], then SubInfo[stages][4], then the barriers
    static constexpr int kInfoAt = kStages * kStageBytes;
    static constexpr int kBarsAt = kInfoAt + kStages * kWarps * (int)sizeof(SubInfo);
    static constexpr int kAbortAt = kBarsAt + 16 * kStages;
    static constexpr int kBytes = kAbortAt + 16;
    // the joining of the warps reuses the ring: [warps][rows][D + 4] sums, maxima, sums of weights
    static constexpr int kLd = D + 4;
    static_assert(kWarps * kRows * (kLd + 2) * 4 <= kInfoAt, "");
};

// Few query rows: a tile of 16 rows over a share of its tokens.  One warp
// copies whole pages' parts into a ring of stages of 64 tokens (their codes
// lie in one piece for a page and head), four take 16 tokens of each stage
// with all rows.  Bound by reading the codes; at 64 sequences of up to 8192
// tokens, 8 x 8 heads of 128, the ring's two CTAs per SM keep HBM busy.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 2) kv_attention_kernel(const AttnArgs a) {
    using R = Ring<D>;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t ring = smem_u32(smem), bars = ring + R::kBarsAt;   // full[stages], empty[stages]
    SubInfo* info = reinterpret_cast<SubInfo*>(smem + R::kInfoAt);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + R::kAbortAt);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int64_t u = blockIdx.x / a.splits;
    const int h = blockIdx.y, split = blockIdx.x % a.splits;
    const bool cluster = a.splits > 1 && !a.partial;
    Tile tile;
    // A cluster's CTAs have one tile: they leave here together or not at all.
    if (!tile.find(a, u, threadIdx.x == 0 && h == 0 && split == 0) || (!cluster && split >= tile.active)) return;
    const int step_begin = min(tile.steps, split * tile.per);
    const int steps = min(tile.steps, step_begin + tile.per) - step_begin;
    const int64_t tok_begin = tile.tok0 + (int64_t)step_begin * kStep;
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
    float* s_m = s_o + kWarps * kRows * R::kLd;                      // [warps][rows]
    float* s_l = s_m + kWarps * kRows;
    if (warp == kWarps) {
        // ---- copies: lane i looks up 16 tokens, for 32 of them at a time ----
        const int32_t* table = a.b.table + tile.seq * a.b.width;
        const int log2 = a.c.page_log2, chunk = min(kStep, 1 << log2);   // tokens of one copy
        [[maybe_unused]] const int64_t code_bytes = a.c.pages * a.c.heads * ((int64_t)D << log2);
        SubInfo mine = {};
        int64_t from = 0;
        uint32_t phase = 0;
        int stage = 0, issued = 0;
        for (int s = 0; s < steps; ++s) {
            if (s % 8 == 0) {
                const int64_t tok = tok_begin + (int64_t)s * kStep + lane * kSub;
                bool live = tok < tile.hi;
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
            int ok = 1;
            if (lane == 0) ok = mbar_wait(bars + 8 * (R::kStages + stage), phase ^ 1u, abort_flag, a.err, kWaitLimitNs);
            if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) break;
            const int sub = lane - s % 8 * kWarps;   // this lane's part of the stage, if it has one
            const bool here = sub >= 0 && sub < kWarps;
            // the first 16 tokens of a page's part fetch all of it
            bool copies = here && mine.live && sub * kSub % chunk == 0;
            if (copies) copies = GEMM_DBG_OK(a.c.k + from, a.c.k, code_bytes, chunk * D) && GEMM_DBG_OK(a.c.v + from, a.c.v, code_bytes, chunk * D);
            if (here) info[stage * kWarps + sub] = mine;
            const int parts = __popc(__ballot_sync(0xFFFFFFFFu, copies));
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(bars + 8 * stage, (uint32_t)(parts * 2 * chunk * D));
            __syncwarp();
            if (copies) {
                const uint32_t to = ring + stage * R::kStageBytes + sub * kSub * D;
                bulk_load(to, a.c.k + from, chunk * D, bars + 8 * stage);
                bulk_load(to + kStep * D, a.c.v + from, chunk * D, bars + 8 * stage);
            }
            ++issued;
            if (++stage == R::kStages) stage = 0, phase ^= 1u;
        }
        // Copies in flight land before the CTA may leave or reuse the ring.
        for (int s = max(0, issued - R::kStages); s < issued; ++s) {
            if (lane == 0) {
                const uint32_t bar = bars + 8 * (s % R::kStages), parity = (uint32_t)(s / R::kStages) & 1u;
                const uint64_t t0 = global_ns();
                while (!mbar_try_wait(bar, parity))
                    if (global_ns() - t0 > kWaitLimitNs) {
                        atomicOr(a.err, kErrTimeout);
                        break;
                    }
            }
        }
        __syncwarp();
        __syncthreads();   // the ring is free
        __syncthreads();   // the warps' results are in it
    } else {
        // Q rows g and g + 8 as A fragments.  A lane's part of a row is 16
        // neighbours of each 64: its k of four instructions, in the order in
        // which its 16 bytes of a key row hold them.  bfloat16 rows are brought
        // to [1, 2) by a power of two (exact, but for elements under 2^-14 of the
        // row's largest, whose error stays under 2^-25 of it) to be binary16.
        uint32_t qf[D / 16][4];
        float row_scale[2];
        int64_t row_lo[2], row_hi[2];
        [[maybe_unused]] const int64_t q_bytes =
            ((a.b.rows - 1) * a.Q.row + (a.q_heads - 1) * a.Q.head + D) * (int64_t)sizeof(T);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t r = tile.r0 + g + 8 * i;
            const bool live = r < tile.nrows;
            const T* p = static_cast<const T*>(a.Q.p) + (tile.row0 + (live ? r / a.share : 0)) * a.Q.row +
                         (h * a.share + (live ? r % a.share : 0)) * a.Q.head;
            Eight<T> x[D / 64][2] = {};
            float top = 0.0f;
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const T* pe = p + 64 * j + 16 * t + 8 * e;
                    if (live && GEMM_DBG_OK(pe, a.Q.p, q_bytes, 16)) x[j][e] = load_eight(pe, a.q_vec);
                }
            float up = 1.0f, down = 1.0f;
            if constexpr (!std::is_same<T, __half>::value) {
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
            row_scale[i] = a.scale_log2 * up;
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const Eight<T>& e = x[j][s / 2];
                    const int o = 4 * (s % 2);
                    qf[4 * j + s][i] = pack2<__half>(e.at(o) * down, e.at(o + 1) * down);
                    qf[4 * j + s][2 + i] = pack2<__half>(e.at(o + 2) * down, e.at(o + 3) * down);
                }
            row_lo[i] = tile.row_lo(a, r);
            row_hi[i] = tile.row_hi(a, r);
        }
        // tokens that every row of the tile sees (rows past the last one see none)
        const int64_t full_lo = tile.row_lo(a, tile.r0 + kRows - 1);
        const int64_t full_hi = tile.r0 + kRows <= tile.nrows ? tile.row_hi(a, tile.r0) : 0;

        constexpr int NT = D / 8;      // column tiles of the output
        float o[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
        float m[2] = {kNegInf, kNegInf}, l[2] = {0.0f, 0.0f}, ref = 0.0f;

        uint32_t phase = 0;
        int stage = 0;
        for (int s = 0; s < steps; ++s) {
            if (!mbar_wait(bars + 8 * stage, phase, abort_flag, a.err, kWaitLimitNs)) break;
            const SubInfo in = info[stage * kWarps + warp];
            const uint32_t kat = ring + stage * R::kStageBytes + warp * kSub * D, vat = kat + kStep * D;
            if (in.live) {
                const int64_t tok = tok_begin + (int64_t)s * kStep + warp * kSub;
                float sc[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    float part[2][4] = {};
#pragma unroll
                    for (int j = 0; j < D / 64; ++j) {
                        const uint4 w = lds128(kat + (8 * n + g) * D + 64 * j + 16 * t);
                        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t(&f)[4] = qf[4 * j + k];
                            mma_16816<__half>(part[k & 1], f[0], f[1], f[2], f[3], codes01(ws[k]), codes23(ws[k]));
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[n][e] = part[0][e] + part[1][e];
                }
                uint32_t vw[4][D / 32];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t at = vat + (8 * (i >> 1) + 2 * t + (i & 1)) * D + g * (D / 8);
                    if constexpr (D == 128) {
                        const uint4 w = lds128(at);
                        vw[i][0] = w.x, vw[i][1] = w.y, vw[i][2] = w.z, vw[i][3] = w.w;
                    } else {
                        const uint2 w = lds64(at);
                        vw[i][0] = w.x, vw[i][1] = w.y;
                    }
                }
                const bool all = tok >= full_lo && tok + kSub <= full_hi;
                const float f0 = row_scale[0] * in.ks, f1 = row_scale[1] * in.ks;
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x = sc[n][e] * (e < 2 ? f0 : f1);
                        if (!all) {
                            const int64_t j = tok + 8 * n + 2 * t + (e & 1);
                            if (j < row_lo[e >> 1] || j >= row_hi[e >> 1]) x = kNegInf;
                        }
                        sc[n][e] = x;
                    }
                float top[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    top[i] = fmaxf(fmaxf(sc[0][2 * i], sc[0][2 * i + 1]), fmaxf(sc[1][2 * i], sc[1][2 * i + 1]));
                    top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 1));
                    top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 2));
                }
                // The sums so far are brought to a new maximum, or a new largest
                // value scale, only when there is one.
                if (__any_sync(0xFFFFFFFFu, top[0] > m[0] || top[1] > m[1] || in.vs > ref)) {
                    const float nref = fmaxf(ref, in.vs);
                    const float grow = ref == nref ? 1.0f : ref / nref;   // ref = 0 at first: o is still 0
                    float keep[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float nm = fmaxf(m[i], top[i]);
                        keep[i] = exp2_approx(m[i] - (nm == kNegInf ? 0.0f : nm));
                        m[i] = nm;
                        l[i] *= keep[i];
                        keep[i] *= grow;
                    }
                    ref = nref;
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        o[i][0] *= keep[0], o[i][1] *= keep[0];
                        o[i][2] *= keep[1], o[i][3] *= keep[1];
                    }
                }
                // A page's value scale relative to the largest so far, times 2^15:
                // the weight is a binary16 of at most 2^15, normal down to 2^-29 of
                // the largest possible.
                const float f = ref == 0.0f && in.vs == 0.0f ? 0.0f : in.vs / ref * kPScale;
                const float base[2] = {m[0] == kNegInf ? 0.0f : m[0], m[1] == kNegInf ? 0.0f : m[1]};
                uint32_t pf[4];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    float p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float x = sc[n][e];
                        const float w = exp2_approx(x - base[e >> 1]);
                        l[e >> 1] += w;
                        p[e] = x == kNegInf ? 0.0f : w * f;   // where f is NaN, only a seen token's
                    }
                    pf[2 * n] = pack2<__half>(p[0], p[1]);
                    pf[2 * n + 1] = pack2<__half>(p[2], p[3]);
                }
#pragma unroll
                for (int e = 0; e < D / 32; ++e) {
                    const uint32_t a01 = __byte_perm(vw[0][e], vw[1][e], 0x5140), a23 = __byte_perm(vw[0][e], vw[1][e], 0x7362);
                    const uint32_t b01 = __byte_perm(vw[2][e], vw[3][e], 0x5140), b23 = __byte_perm(vw[2][e], vw[3][e], 0x7362);
                    mma_16816<__half>(o[4 * e], pf[0], pf[1], pf[2], pf[3], codes01(a01), codes01(b01));
                    mma_16816<__half>(o[4 * e + 1], pf[0], pf[1], pf[2], pf[3], codes23(a01), codes23(b01));
                    mma_16816<__half>(o[4 * e + 2], pf[0], pf[1], pf[2], pf[3], codes01(a23), codes01(b23));
                    mma_16816<__half>(o[4 * e + 3], pf[0], pf[1], pf[2], pf[3], codes23(a23), codes23(b23));
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bars + 8 * (R::kStages + stage));
            if (++stage == R::kStages) stage = 0, phase ^= 1u;
        }
        __syncthreads();   // the ring is free: every copy has landed and been used

        // Join the warps: each has a maximum, a sum and unnormalised outputs.
        const float unit = ref / kPScale;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 1);
            l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 2);
            if (t == 0) s_m[warp * kRows + g + 8 * i] = m[i], s_l[warp * kRows + g + 8 * i] = l[i];
            float* row = s_o + (warp * kRows + g + 8 * i) * R::kLd;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                row[2 * t * NT + n] = o[n][2 * i] * unit;
                row[(2 * t + 1) * NT + n] = o[n][2 * i + 1] * unit;
            }
        }
        __syncthreads();
    }

    [[maybe_unused]] const int64_t o_bytes =
        ((a.b.rows - 1) * a.O.row + (a.q_heads - 1) * a.O.head + D) * (int64_t)sizeof(T);
    const int rows = (int)(tile.nrows - tile.r0 < kRows ? tile.nrows - tile.r0 : kRows);
    const bool whole = a.splits == 1 || (!cluster && tile.active == 1);
    float* part = a.partial ? a.partial + ((u * a.c.heads + h) * a.splits + split) * (kRows * (D + 2)) : nullptr;
    for (int i = threadIdx.x; i < rows * D; i += kThreads) {
        const int r = i / D, d = i % D;
        float top = s_m[r];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_m[w * kRows + r]);
        const float from = top == kNegInf ? 0.0f : top;
        float sum = 0.0f, acc = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = exp2_approx(s_m[w * kRows + r] - from);
            sum = fmaf(f, s_l[w * kRows + r], sum);
            acc = fmaf(f, s_o[(w * kRows + r) * R::kLd + d], acc);
        }
        if (whole) {
            T* dst = out_row<T>(a, tile, h, tile.r0 + r) + d;
            if (GEMM_DBG_OK(dst, a.O.p, o_bytes, sizeof(T))) *dst = from_float<T>(sum == 0.0f ? 0.0f : acc / sum);
        } else if (cluster) {
            s_o[r * R::kLd + d] = acc;   // warp 0's place: read by this thread alone so far
            if (d == 0) {
                float* ml = s_l + kWarps * kRows + 2 * r;
                ml[0] = top, ml[1] = sum;
            }
        } else {
            part[i] = acc;
            if (d == 0) part[kRows * D + 2 * r] = top, part[kRows * D + 2 * r + 1] = sum;
        }
    }
    if (!cluster) return;
    // The cluster's CTAs each join a share of the results, in split order.
    cluster_sync();
    const int share = (rows * D + a.splits - 1) / a.splits;
    for (int i = split * share + threadIdx.x; i < min(rows * D, (split + 1) * share); i += kThreads) {
        const int r = i / D, d = i % D;
        const uint32_t ml = smem_u32(s_l + kWarps * kRows + 2 * r), at = smem_u32(s_o + r * R::kLd + d);
        float tops[kMaxCluster], sums[kMaxCluster], accs[kMaxCluster], top = kNegInf;
#pragma unroll
        for (int s = 0; s < kMaxCluster; ++s) {
            if (s >= tile.active) break;
            tops[s] = ld_cluster_f32(mapa_shared(ml, s));
            sums[s] = ld_cluster_f32(mapa_shared(ml + 4, s));
            accs[s] = ld_cluster_f32(mapa_shared(at, s));
            top = fmaxf(top, tops[s]);
        }
        const float from = top == kNegInf ? 0.0f : top;
        float sum = 0.0f, acc = 0.0f;
#pragma unroll
        for (int s = 0; s < kMaxCluster; ++s) {
            if (s >= tile.active) break;
            const float f = exp2_approx(tops[s] - from);
            sum = fmaf(f, sums[s], sum);
            acc = fmaf(f, accs[s], acc);
        }
        T* dst = out_row<T>(a, tile, h, tile.r0 + r) + d;
        if (GEMM_DBG_OK(dst, a.O.p, o_bytes, sizeof(T))) *dst = from_float<T>(sum == 0.0f ? 0.0f : acc / sum);
    }
    cluster_sync();   // no CTA leaves while another reads its results
}

// Joins the splits of one row of a tile, in order: four threads share an
// output element's splits.
template <typename T, int D>
__global__ void __launch_bounds__(4 * D) kv_join_kernel(const AttnArgs a) {
    __shared__ float s_acc[4][D], s_sum[4];
    const int64_t u = blockIdx.x;
    const int h = blockIdx.y, r = blockIdx.z, d = threadIdx.x % D, q = threadIdx.x / D;
    Tile tile;
    if (!tile.find(a, u, false) || tile.active == 1 || tile.r0 + r >= tile.nrows) return;
    constexpr int64_t kSlot = kRows * (D + 2);
    const float* part = a.partial + (u * a.c.heads + h) * a.splits * kSlot;
    const float* ml = part + kRows * D + 2 * r;
    float top = kNegInf;
    for (int s = threadIdx.x % 32; s < tile.active; s += 32) top = fmaxf(top, ml[s * kSlot]);
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, i));
    const float from = top == kNegInf ? 0.0f : top;
    const int share = (tile.active + 3) / 4, end = min(tile.active, (q + 1) * share);
    float sum = 0.0f, acc = 0.0f;
#pragma unroll 4
    for (int s = q * share; s < end; ++s) {
        const float f = exp2_approx(ml[s * kSlot] - from);
        sum = fmaf(f, ml[s * kSlot + 1], sum);
        acc = fmaf(f, part[s * kSlot + r * D + d], acc);
    }
    s_acc[q][d] = acc;
    if (d == 0) s_sum[q] = sum;
    __syncthreads();
    if (q != 0) return;
    [[maybe_unused]] const int64_t o_bytes =
        ((a.b.rows - 1) * a.O.row + (a.q_heads - 1) * a.O.head + D) * (int64_t)sizeof(T);
    acc = ((s_acc[0][d] + s_acc[1][d]) + s_acc[2][d]) + s_acc[3][d];
    sum = ((s_sum[0] + s_sum[1]) + s_sum[2]) + s_sum[3];
    T* dst = out_row<T>(a, tile, h, tile.r0 + r) + d;
    if (GEMM_DBG_OK(dst, a.O.p, o_bytes, sizeof(T))) *dst = from_float<T>(sum == 0.0f ? 0.0f : acc / sum);
}

template <typename T, int D>
cudaError_t launch(const AttnArgs& a, const KvPlan& plan, int* launches, cudaStream_t stream) {
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
    cudaError_t e = cudaLaunchKernelEx(&cfg, kv_attention_kernel<T, D>, a);
    *launches = 1;
    if (e == cudaSuccess && a.partial) {
        kv_join_kernel<T, D><<<dim3((unsigned)plan.units, (unsigned)a.c.heads, kRows), 4 * D, 0, stream>>>(a);
        e = cudaGetLastError();
        *launches = 2;
    }
    return e;
}

template <typename T, int D>
cudaError_t allow_smem() {
    return cudaFuncSetAttribute(kv_attention_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Ring<D>::kBytes);
}

}  // namespace

LIBGEMM_DEBUG_READER(kv_attention_debug_flags)

cudaError_t kv_attention_setup() {
    cudaError_t e = allow_smem<__nv_bfloat16, 64>();
    if (e == cudaSuccess) e = allow_smem<__nv_bfloat16, 128>();
    if (e == cudaSuccess) e = allow_smem<__half, 64>();
    if (e == cudaSuccess) e = allow_smem<__half, 128>();
    return e;
}

// Tiles of rows that fill an eighth of the GPU's CTA slots or more, or whose
// tokens are few, have their tokens shared over a cluster (joined through
// distributed shared memory, no second launch): four rounds of CTAs, as
// sequences differ in length.  Fewer tiles over long sequences are shared over
// one round of CTAs and joined by a second kernel.
KvPlan kv_plan(const KvView& c, const KvBatch& b, int q_heads, int64_t window, int num_sms) {
    const int64_t share = q_heads / c.heads, tiles = b.rows * share / kRows;
    KvPlan p;
    p.units = tiles + b.sequences;
    int64_t longest = b.width << c.page_log2;
    if (window > 0 && window + 2 * kStep < longest) longest = window + 2 * kStep;
    const int64_t have = (tiles > b.sequences ? tiles : b.sequences) * c.heads, slots = 2 * (int64_t)num_sms;
    const int64_t most = (longest + kStep * kMinSteps - 1) / (kStep * kMinSteps);
    const bool cluster = most <= 8 * kMaxCluster || have * kMaxCluster >= slots;
    int64_t splits = cluster ? (4 * slots + have - 1) / have : slots / have;
    if (splits > most) splits = most;
    if (cluster && splits > kMaxCluster) splits = kMaxCluster;
    p.splits = (int)(splits < 1 ? 1 : splits);
    p.scratch_bytes = p.splits > kMaxCluster ? p.units * c.heads * p.splits * (kRows * (c.dim + 2) * 4) : 0;
    return p;
}

cudaError_t launch_kv_attention(const KvView& c, const KvRows& Q, const KvRows& O, ElemType type,
                                int q_heads, float scale, bool causal, int64_t window,
                                const KvBatch& b, const KvPlan& plan, void* scratch,
                                unsigned* err, int* launches, cudaStream_t stream) {
    const bool q_vec = (reinterpret_cast<uintptr_t>(Q.p) & 15u) == 0 && Q.row % 8 == 0 && Q.head % 8 == 0;
    const AttnArgs a{c, Q, O, b, q_heads, q_heads / c.heads, scale * 1.44269504088896341f, causal,
                     window, plan.splits, q_vec, static_cast<float*>(scratch), err};
    if (type == ElemType::kBF16)
        return c.dim == 128 ? launch<__nv_bfloat16, 128>(a, plan, launches, stream)
                            : launch<__nv_bfloat16, 64>(a, plan, launches, stream);
    return c.dim == 128 ? launch<__half, 128>(a, plan, launches, stream)
                        : launch<__half, 64>(a, plan, launches, stream);
}

}  // namespace libgemm
