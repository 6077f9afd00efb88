// kv4_attention.cu -- attention of ragged queries over the paged 4-bit cache.
//
// For each query row  o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale * q.k_j
// - m), in one pass over the tokens with the running maximum m and sum.  A warp
// has one row: its lanes take a token each for the scores, and then each a
// thirty-second of the dimensions for the values.
#include "kv_attention.cuh"

namespace libgemm {
namespace {

constexpr int kThreads = 128;

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv4_attention_kernel(const AttnArgs a) {
    constexpr int kEach = D / 32;
    __shared__ float s_q[kThreads / 32][D];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + warp;
    const int head = blockIdx.y, h = head / a.share;
    const Starts starts{a.b.starts, a.b.sequences, a.b.rows};
    if (blockIdx.x == 0 && head == 0) starts.check(a.err);
    if (row >= a.b.rows) return;
    const int seq = last_not_above(a.b.sequences, row, row, [&](int i) { return starts.at(i); });
    if (!starts.good(seq)) return;
    const int64_t row0 = starts.at(seq), count = starts.at(seq + 1) - row0;
    if (row < row0 || row >= row0 + count) return;
    int len = __ldg(a.b.at + seq);
    if (len < 0 || len > (a.b.width << a.c.page_log2)) {
        if (lane == 0) atomicOr(a.err, kErrIndex);
        len = 0;
    }
    const int p = len - (int)(count - (row - row0));
    const int hi = p < 0 ? 0 : a.causal ? p + 1 : len, lo = a.window > 0 && p >= a.window ? p - a.window + 1 : 0;
    const T* q = static_cast<const T*>(a.Q.p) + row * a.Q.row + head * a.Q.head;
    for (int d = lane; d < D; d += 32) s_q[warp][d] = (float)q[d];
    __syncwarp();
    const int page = 1 << a.c.page_log2;
    const int32_t* table = a.b.table + seq * a.b.width;
    float m = kLowest, l = 0.0f, o[kEach] = {};
    for (int tok0 = lo / 32 * 32; tok0 < hi; tok0 += 32) {
        const int tok = tok0 + lane;
        float s = kNegInf, vs = 0.0f;
        const uint8_t* codes = nullptr;      // of the values of this token's block of 16
        if (tok >= lo && tok < hi) {
            const int64_t at = __ldg(table + (tok >> a.c.page_log2));
            if (at < 0 || at >= a.c.pages) {
                atomicOr(a.err, kErrIndex);
            } else {
                const uint8_t* record = a.c.data + (at * a.c.heads + h) * a.c.record();
                const int in = tok & (page - 1);
                const uint16_t* scales = reinterpret_cast<const uint16_t*>(record + page * D);
                const float ks = __uint_as_float((uint32_t)scales[in] << 16);
                vs = __uint_as_float((uint32_t)scales[page + in] << 16);
                float dot = 0.0f;
                for (int t = 0; t < 4; ++t)
                    for (int i = 0; i < D / 32; ++i) {
                        const uint32_t w = *reinterpret_cast<const uint32_t*>(record + in * (D / 2) + t * (D / 8) + 4 * i);
                        for (int e = 0; e < 8; ++e)
                            dot = fmaf(s_q[warp][32 * i + 8 * t + e], (float)((int)(w >> (4 * e) & 15u) - 8), dot);
                    }
                s = dot * ks * a.scale_log2;
                codes = record + page * (D / 2) + in / 16 * (8 * D);
            }
        }
        float top = s;
        for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, i));
        top = fmaxf(top, m);
        const float keep = exp2_approx(m - top), w = codes ? exp2_approx(s - top) : 0.0f;
        m = top;
        float sum = w;
        for (int i = 16; i > 0; i >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, i);
        l = fmaf(l, keep, sum);
        for (int e = 0; e < kEach; ++e) o[e] *= keep;
        for (int j = 0; j < 32; ++j) {
            const float wv = __shfl_sync(0xFFFFFFFFu, w * vs, j);
            const uint8_t* from = reinterpret_cast<const uint8_t*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(codes), j));
            if (!from) continue;
            for (int e = 0; e < kEach; ++e) {
                const int d = lane + 32 * e, t = (tok0 + j) % 16;
                const int at = t / 8 * (4 * D) + (4 * (d % 64 / 8) + t % 8 / 2) * (D / 8) + d / 64 * 8 + d % 8 / 4 * 4 + t % 2 * 2 + d % 4 / 2;
                o[e] = fmaf(wv, (float)((int)(from[at] >> (4 * (d % 2)) & 15) - 8), o[e]);
            }
        }
    }
    T* out = static_cast<T*>(a.O.p) + row * a.O.row + head * a.O.head;
    for (int e = 0; e < kEach; ++e) out[lane + 32 * e] = from_float<T>(l == 0.0f ? 0.0f : o[e] / l);
}

}  // namespace

LIBGEMM_DEBUG_READER(kv4_attention_debug_flags)

cudaError_t launch_kv4_few(const AttnArgs& a, ElemType type, const KvPlan&, cudaStream_t stream) {
    const dim3 grid((unsigned)((a.b.rows + kThreads / 32 - 1) / (kThreads / 32)), (unsigned)a.q_heads);
    if (type == ElemType::kBF16 && a.c.dim == 128) kv4_attention_kernel<__nv_bfloat16, 128><<<grid, kThreads, 0, stream>>>(a);
    else if (type == ElemType::kBF16) kv4_attention_kernel<__nv_bfloat16, 64><<<grid, kThreads, 0, stream>>>(a);
    else if (a.c.dim == 128) kv4_attention_kernel<__half, 128><<<grid, kThreads, 0, stream>>>(a);
    else kv4_attention_kernel<__half, 64><<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace libgemm
