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
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 32;        // tokens a warp takes at once
constexpr int kMinSteps = 8;     // steps of a split, at least
constexpr float kNegInf = -INFINITY;
constexpr float kPScale = 32768.0f;   // weights enter the second product times 2^15

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
    int splits;
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

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv_attention_kernel(const AttnArgs a) {
    __shared__ float s_o[kWarps][kRows][D + 4];
    __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int64_t u = blockIdx.x;
    const int h = blockIdx.y, split = blockIdx.z;
    Tile tile;
    if (!tile.find(a, u, threadIdx.x == 0 && h == 0 && split == 0) || split >= tile.active) return;
    const int step_begin = split * tile.per;
    const int step_end = min(tile.steps, step_begin + tile.per);

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
        float x[D / 64][16];
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const T* pe = p + 64 * j + 16 * t + e;
                x[j][e] = live && GEMM_DBG_OK(pe, a.Q.p, q_bytes, sizeof(T)) ? to_float(*pe) : 0.0f;
                top = fmaxf(top, fabsf(x[j][e]));
            }
        float up = 1.0f, down = 1.0f;
        if constexpr (sizeof(T) == 2 && !std::is_same<T, __half>::value) {
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
                qf[4 * j + s][i] = pack2<__half>(x[j][4 * s] * down, x[j][4 * s + 1] * down);
                qf[4 * j + s][2 + i] = pack2<__half>(x[j][4 * s + 2] * down, x[j][4 * s + 3] * down);
            }
        row_lo[i] = tile.row_lo(a, r);
        row_hi[i] = tile.row_hi(a, r);
    }
    // tokens that every row of the tile sees
    const int64_t full_lo = tile.row_lo(a, tile.r0 + kRows - 1), full_hi = tile.r0 + kRows <= tile.nrows ? tile.row_hi(a, tile.r0) : 0;

    constexpr int NT = D / 8;      // column tiles of the output
    float o[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    float m[2] = {kNegInf, kNegInf}, l[2] = {0.0f, 0.0f}, ref = 0.0f;
    const int32_t* table = a.b.table + tile.seq * a.b.width;
    [[maybe_unused]] const int64_t code_bytes = a.c.pages * a.c.heads * ((int64_t)D << a.c.page_log2);

    for (int step = step_begin + warp; step < step_end; step += kWarps) {
        const int64_t tok = tile.tok0 + (int64_t)step * kStep;
        uint4 kw[4][D / 64];
        uint32_t vw[2][4][D / 32];
        float ks[2] = {0.0f, 0.0f}, vs[2] = {0.0f, 0.0f};
        bool live[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int64_t ts = tok + 16 * s;
            live[s] = ts < tile.hi;
            int64_t page = live[s] ? __ldg(table + (ts >> a.c.page_log2)) : 0;
            if (live[s] && (page < 0 || page >= a.c.pages)) {
                if (lane == 0) atomicOr(a.err, kErrIndex);
                live[s] = false;
            }
            const int64_t ph = page * a.c.heads + h;
            const int64_t base = ((ph << a.c.page_log2) + (ts & ((1 << a.c.page_log2) - 1))) * D;
            if (live[s]) ks[s] = __ldg(a.c.ks + ph), vs[s] = __ldg(a.c.vs + ph);
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int j = 0; j < D / 64; ++j) {
                    const uint8_t* p = a.c.k + base + (8 * n + g) * D + 64 * j + 16 * t;
                    kw[2 * s + n][j] = make_uint4(0, 0, 0, 0);
                    if (live[s] && GEMM_DBG_OK(p, a.c.k, code_bytes, 16))
                        kw[2 * s + n][j] = __ldcs(reinterpret_cast<const uint4*>(p));
                }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint8_t* p = a.c.v + base + (8 * (i >> 1) + 2 * t + (i & 1)) * D + g * (D / 8);
#pragma unroll
                for (int e = 0; e < D / 32; ++e) vw[s][i][e] = 0x80808080u;
                if (live[s] && GEMM_DBG_OK(p, a.c.v, code_bytes, D / 8)) {
                    if constexpr (D == 128) {
                        const uint4 w = __ldcs(reinterpret_cast<const uint4*>(p));
                        vw[s][i][0] = w.x, vw[s][i][1] = w.y, vw[s][i][2] = w.z, vw[s][i][3] = w.w;
                    } else {
                        const uint2 w = __ldcs(reinterpret_cast<const uint2*>(p));
                        vw[s][i][0] = w.x, vw[s][i][1] = w.y;
                    }
                }
            }
        }
        float sc[4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.0f;
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                const uint32_t ws[4] = {kw[n][j].x, kw[n][j].y, kw[n][j].z, kw[n][j].w};
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const uint32_t(&f)[4] = qf[4 * j + s];
                    mma_16816<__half>(sc[n], f[0], f[1], f[2], f[3], codes01(ws[s]), codes23(ws[s]));
                }
            }
        }
        const bool all = tok >= full_lo && tok + kStep <= full_hi && live[0] && live[1];
        float top[2] = {kNegInf, kNegInf};
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = e >> 1;
                float x = sc[n][e] * (row_scale[i] * ks[n >> 1]);
                if (!all) {
                    const int64_t j = tok + 8 * n + 2 * t + (e & 1);
                    if (j < row_lo[i] || j >= row_hi[i] || !live[n >> 1]) x = kNegInf;
                }
                sc[n][e] = x;
                top[i] = fmaxf(top[i], x);
            }
        const float nref = fmaxf(ref, fmaxf(vs[0], vs[1]));
        const float grow = ref == nref ? 1.0f : ref / nref;   // ref = 0 at first: o is still 0
        float base[2], keep[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 1));
            top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 2));
            const float nm = fmaxf(m[i], top[i]);
            base[i] = nm == kNegInf ? 0.0f : nm;
            keep[i] = exp2_approx(m[i] - base[i]);
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
        // A page's value scale relative to the largest so far, times 2^15:
        // the weight is a binary16 of at most 2^15, normal down to 2^-29 of
        // the largest possible.
        uint32_t pf[2][4];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const float f = ref == 0.0f && vs[s] == 0.0f ? 0.0f : vs[s] / ref * kPScale;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                float p[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x = sc[2 * s + n][e];
                    const float w = exp2_approx(x - base[e >> 1]);
                    l[e >> 1] += w;
                    p[e] = x == kNegInf ? 0.0f : w * f;
                }
                pf[s][2 * n] = pack2<__half>(p[0], p[1]);
                pf[s][2 * n + 1] = pack2<__half>(p[2], p[3]);
            }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {
                const uint32_t a01 = __byte_perm(vw[s][0][e], vw[s][1][e], 0x5140), a23 = __byte_perm(vw[s][0][e], vw[s][1][e], 0x7362);
                const uint32_t b01 = __byte_perm(vw[s][2][e], vw[s][3][e], 0x5140), b23 = __byte_perm(vw[s][2][e], vw[s][3][e], 0x7362);
                const uint32_t(&f)[4] = pf[s];
                mma_16816<__half>(o[4 * e], f[0], f[1], f[2], f[3], codes01(a01), codes01(b01));
                mma_16816<__half>(o[4 * e + 1], f[0], f[1], f[2], f[3], codes23(a01), codes23(b01));
                mma_16816<__half>(o[4 * e + 2], f[0], f[1], f[2], f[3], codes01(a23), codes01(b23));
                mma_16816<__half>(o[4 * e + 3], f[0], f[1], f[2], f[3], codes23(a23), codes23(b23));
            }
    }

    // Join the warps: each has a maximum, a sum and unnormalised outputs.
    const float unit = ref / kPScale;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 1);
        l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 2);
        if (t == 0) s_m[warp][g + 8 * i] = m[i], s_l[warp][g + 8 * i] = l[i];
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        s_o[warp][g][2 * t * NT + i] = o[i][0] * unit;
        s_o[warp][g][(2 * t + 1) * NT + i] = o[i][1] * unit;
        s_o[warp][g + 8][2 * t * NT + i] = o[i][2] * unit;
        s_o[warp][g + 8][(2 * t + 1) * NT + i] = o[i][3] * unit;
    }
    __syncthreads();
    [[maybe_unused]] const int64_t o_bytes =
        ((a.b.rows - 1) * a.O.row + (a.q_heads - 1) * a.O.head + D) * (int64_t)sizeof(T);
    const int64_t slot = (u * a.c.heads + h) * a.splits + split;
    float* part = a.partial + slot * (kRows * (D + 2));
    for (int i = threadIdx.x; i < kRows * D; i += kThreads) {
        const int r = i / D, d = i % D;
        if (tile.r0 + r >= tile.nrows) break;
        float top = s_m[0][r];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_m[w][r]);
        const float from = top == kNegInf ? 0.0f : top;
        float sum = 0.0f, acc = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = exp2_approx(s_m[w][r] - from);
            sum = fmaf(f, s_l[w][r], sum);
            acc = fmaf(f, s_o[w][r][d], acc);
        }
        if (tile.active == 1) {
            T* dst = out_row<T>(a, tile, h, tile.r0 + r) + d;
            if (GEMM_DBG_OK(dst, a.O.p, o_bytes, sizeof(T))) *dst = from_float<T>(sum == 0.0f ? 0.0f : acc / sum);
        } else {
            part[i] = acc;
            if (d == 0) part[kRows * D + 2 * r] = top, part[kRows * D + 2 * r + 1] = sum;
        }
    }
}

// Joins the splits of a tile, in order.
template <typename T, int D>
__global__ void __launch_bounds__(D) kv_join_kernel(const AttnArgs a) {
    const int64_t u = blockIdx.x;
    const int h = blockIdx.y, d = threadIdx.x;
    Tile tile;
    if (!tile.find(a, u, false) || tile.active == 1) return;
    [[maybe_unused]] const int64_t o_bytes =
        ((a.b.rows - 1) * a.O.row + (a.q_heads - 1) * a.O.head + D) * (int64_t)sizeof(T);
    const float* part = a.partial + (u * a.c.heads + h) * a.splits * (kRows * (D + 2));
    for (int r = 0; r < kRows && tile.r0 + r < tile.nrows; ++r) {
        float top = kNegInf;
        for (int s = 0; s < tile.active; ++s) top = fmaxf(top, part[s * (kRows * (D + 2)) + kRows * D + 2 * r]);
        const float from = top == kNegInf ? 0.0f : top;
        float sum = 0.0f, acc = 0.0f;
        for (int s = 0; s < tile.active; ++s) {
            const float* p = part + s * (kRows * (D + 2));
            const float f = exp2_approx(p[kRows * D + 2 * r] - from);
            sum = fmaf(f, p[kRows * D + 2 * r + 1], sum);
            acc = fmaf(f, p[r * D + d], acc);
        }
        T* dst = out_row<T>(a, tile, h, tile.r0 + r) + d;
        if (GEMM_DBG_OK(dst, a.O.p, o_bytes, sizeof(T))) *dst = from_float<T>(sum == 0.0f ? 0.0f : acc / sum);
    }
}

template <typename T, int D>
cudaError_t launch(const AttnArgs& a, const KvPlan& plan, int* launches, cudaStream_t stream) {
    const dim3 grid((unsigned)plan.units, (unsigned)a.c.heads, (unsigned)plan.splits);
    kv_attention_kernel<T, D><<<grid, kThreads, 0, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    *launches = 1;
    if (e == cudaSuccess && plan.splits > 1) {
        kv_join_kernel<T, D><<<dim3(grid.x, grid.y), D, 0, stream>>>(a);
        e = cudaGetLastError();
        *launches = 2;
    }
    return e;
}

}  // namespace

LIBGEMM_DEBUG_READER(kv_attention_debug_flags)

KvPlan kv_plan(const KvView& c, const KvBatch& b, int q_heads, int64_t window, int num_sms) {
    const int64_t share = q_heads / c.heads, tiles = b.rows * share / kRows;
    KvPlan p;
    p.units = tiles + b.sequences;
    int64_t longest = b.width << c.page_log2;
    if (window > 0 && window + 2 * kStep < longest) longest = window + 2 * kStep;
    const int64_t have = (tiles > b.sequences ? tiles : b.sequences) * c.heads;
    int64_t splits = (3 * (int64_t)num_sms + have - 1) / have;
    const int64_t most = (longest + kStep * kMinSteps - 1) / (kStep * kMinSteps);
    if (splits > most) splits = most;
    p.splits = (int)(splits < 1 ? 1 : splits > 512 ? 512 : splits);
    p.scratch_bytes = p.splits > 1 ? p.units * c.heads * p.splits * (kRows * (c.dim + 2) * 4) : 0;
    return p;
}

cudaError_t launch_kv_attention(const KvView& c, const KvRows& Q, const KvRows& O, ElemType type,
                                int q_heads, float scale, bool causal, int64_t window,
                                const KvBatch& b, const KvPlan& plan, void* scratch,
                                unsigned* err, int* launches, cudaStream_t stream) {
    const AttnArgs a{c, Q, O, b, q_heads, q_heads / c.heads, scale * 1.44269504088896341f, causal,
                     window, plan.splits, static_cast<float*>(scratch), err};
    if (type == ElemType::kBF16)
        return c.dim == 128 ? launch<__nv_bfloat16, 128>(a, plan, launches, stream)
                            : launch<__nv_bfloat16, 64>(a, plan, launches, stream);
    return c.dim == 128 ? launch<__half, 128>(a, plan, launches, stream)
                        : launch<__half, 64>(a, plan, launches, stream);
}

}  // namespace libgemm
