// sequences.cu -- what a batch of sequences needs around a paged cache: the plan
// of a step (row offsets, pages, positions, slots) and rotary positions.
#include "kernels.h"
#include "lowbit.cuh"

namespace libgemm {
namespace {

// ---- the plan ------------------------------------------------------------------
// Two launches.  One block sums counts and pages over the sequences, a thread a
// sequence and 1024 at a time, and writes what is one number a sequence; then a
// warp takes 256 rows of a sequence, whose positions and slots follow from the
// sequence's first row and place on the stack alone: the new pages' numbers come off
// the stack, not out of the table, which the same lanes write.
constexpr int kScanThreads = 1024, kFillThreads = 128, kFillRows = 256;

__device__ __forceinline__ int pages_of(int64_t tokens, const StepPlan& p) {   // columns of the table, which is all that are held
    const int64_t n = (tokens + (1 << p.page_log2) - 1) >> p.page_log2;
    return (int)(n < p.width ? n : p.width);
}

__global__ void __launch_bounds__(kScanThreads) plan_scan_kernel(StepPlan p, unsigned* err) {
    __shared__ int64_t s_rows[kScanThreads / 32], s_pages[kScanThreads / 32];
    grid_launch_dependents();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    const int top = *p.available;
    const int height = top < 0 ? 0 : top > p.capacity ? (int)p.capacity : top;
    bool bad = height != top;
    int64_t rows0 = 0, pages0 = 0;   // of the sequences before this round's
    for (int64_t b0 = 0; b0 < p.sequences; b0 += blockDim.x) {
        const int64_t b = b0 + threadIdx.x;
        const bool in = b < p.sequences && GEMM_DBG_OK(p.lengths + b, p.lengths, p.sequences * 4, 4);
        const int length = in ? p.lengths[b] : 0, count = in ? __ldg(p.counts + b) : 0;
        const int held = max(length, 0), added = max(count, 0);
        const int64_t after = (int64_t)held + added;
        bad |= length < 0 || count < 0 || (added > 0 && (after > p.width << p.page_log2 || after > INT32_MAX));
        int64_t rows = added, pages = pages_of(after, p) - pages_of(held, p);   // sums up to this thread's sequence
        for (int i = 1; i < 32; i *= 2) {
            const int64_t r = __shfl_up_sync(0xFFFFFFFFu, rows, i), g = __shfl_up_sync(0xFFFFFFFFu, pages, i);
            if (lane >= i) rows += r, pages += g;
        }
        __syncthreads();   // the last round's sums have been read
        if (lane == 31) s_rows[warp] = rows, s_pages[warp] = pages;
        __syncthreads();
        int64_t rows_all = 0, pages_all = 0;
        for (int w = 0; w < warps; ++w) {
            if (w == warp) rows += rows_all, pages += pages_all;
            rows_all += s_rows[w], pages_all += s_pages[w];
        }
        if (in && GEMM_DBG_OK(p.starts + b, p.starts, (p.sequences + 1) * 4, 4) && GEMM_DBG_OK(p.first + b, p.first, p.sequences * 4, 4)) {
            const int64_t start = rows0 + rows - added, taken = pages0 + pages - (pages_of(after, p) - pages_of(held, p));
            bad |= rows0 + rows > p.tokens || (pages0 + pages > height && taken < pages0 + pages);
            p.starts[b] = (int)(start < p.tokens ? start : p.tokens);
            p.first[b] = held;
            p.heights[b] = (int)(height - taken > INT32_MIN ? height - taken : INT32_MIN);
            p.after[b] = (int)(after < INT32_MAX ? after : INT32_MAX);
        }
        rows0 += rows_all, pages0 += pages_all;
    }
    __syncthreads();   // every thread has read `available`, which may be `left`
    if (threadIdx.x == 0) {
        p.starts[p.sequences] = (int)(rows0 < p.tokens ? rows0 : p.tokens);
        p.heights[p.sequences] = (int)(height - pages0 > INT32_MIN ? height - pages0 : INT32_MIN);
        *p.left = (int)(height > pages0 ? height - pages0 : 0);
    }
    if (bad) atomicOr(err, kErrIndex);
}

__global__ void __launch_bounds__(kFillThreads) plan_fill_kernel(StepPlan p) {
    grid_dependency_wait();
    const int lane = threadIdx.x % 32;
    const int64_t u = (int64_t)blockIdx.x * (kFillThreads / 32) + threadIdx.x / 32;
    // Sequence b's rows are units floor(starts[b] / 256) + b + j, and those past the
    // last sequence's the same of one more.
    const int n = (int)p.sequences;
    auto start = [&](int b) { return (int64_t)p.starts[b]; };
    const int b = last_not_above(n + 1, u, u, [&](int i) { return start(i) / kFillRows + i; });
    const int64_t row0 = start(b), end = b < n ? start(b + 1) : p.tokens;
    const int64_t begin = row0 + (u - row0 / kFillRows - b) * kFillRows;
    if (begin >= end) return;
    const int first = b < n ? p.first[b] : 0, height = b < n ? p.heights[b] : 0, held = pages_of(first, p);
    const int32_t* table = p.table + (int64_t)b * p.width;
    for (int64_t row = begin + lane; row < min(end, begin + kFillRows); row += 32) {
        int position = -1;
        int64_t slot = -1;
        if (b < n) {
            const int64_t at = first + (row - row0);
            position = at <= INT32_MAX ? (int)at : -1;
            const int64_t column = at >> p.page_log2;
            const int in = (int)(at & ((1 << p.page_log2) - 1));
            if (column < p.width && position >= 0) {
                int page;
                if (column < held) {
                    page = table[column];
                } else {   // new, off the stack; its first token writes the table
                    const int64_t from = height - 1 - (column - held);
                    page = from >= 0 && GEMM_DBG_OK(p.free + from, p.free, p.capacity * 4, 4) ? __ldg(p.free + from) : -1;
                    if (in == 0 && GEMM_DBG_OK(table + column, p.table, p.sequences * p.width * 4, 4))
                        p.table[(int64_t)b * p.width + column] = page;
                }
                if (page >= 0) slot = ((int64_t)page << p.page_log2) + in;
            }
        }
        if (!GEMM_DBG_OK(p.positions + row, p.positions, p.tokens * 4, 4) || !GEMM_DBG_OK(p.slots + row, p.slots, p.tokens * 8, 8)) continue;
        p.positions[row] = position;
        p.slots[row] = slot;
    }
}

// ---- rotary positions ------------------------------------------------------------
// A block has some rows with all heads of both operands.  Its threads first make
// the rows' sines and cosines, one a pair, in shared memory: the angle is
// position * turns mod 2^64 in fractions of a turn, one integer product without any
// loss, of which the upper 32 bits become a binary32 half turn count in [-1, 1).  Then
// each thread has one place of a head -- PER elements of either half, or PER
// neighbours -- and goes through rows and heads, so that it reads the sines of a row
// once.
constexpr int kRotaryThreads = 256;

template <typename T>
__device__ __forceinline__ float as_float(T x) {
    if constexpr (std::is_same<T, float>::value) return x;
    else if constexpr (std::is_same<T, __half>::value) return __half2float(x);
    else return __bfloat162float(x);
}

// PER elements as the 16 bytes that hold them, or one.
template <typename T, int PER>
struct Piece {
    float v[PER];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (PER == 1) v[0] = as_float(*p);
        else {
            const uint4 w = *reinterpret_cast<const uint4*>(p);
            const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
            for (int i = 0; i < PER; ++i) v[i] = as_float(e[i]);
        }
    }
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (PER == 1) *p = from_float<T>(v[0]);
        else if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        else *reinterpret_cast<uint4*>(p) = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
    }
};

template <typename T, int PER, bool INTERLEAVED>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const RotaryArgs a, int rows_each, bool inverse, int turned, int places) {
    extern __shared__ float2 s_by[];   // [rows][pairs]: cosine and sine
    const int half = a.part / 2;
    const int64_t row0 = (int64_t)blockIdx.x * rows_each;
    const int rows = (int)(a.rows - row0 < rows_each ? a.rows - row0 : rows_each);
    for (int i = threadIdx.x; i < rows * half; i += kRotaryThreads) {
        const int r = i / half, pair = i % half;
        const int position = __ldg(a.positions + row0 + r);
        const uint64_t turn = (uint64_t)(uint32_t)position * __ldg(a.turns + pair);
        float s, c;
        sincospif((float)(int)(turn >> 32) * 4.656612873077393e-10f, &s, &c);   // 2^-31
        s_by[i] = make_float2(c * a.magnitude, (inverse ? -s : s) * a.magnitude);
    }
    __syncthreads();
    // Places of a head: `turned` that turn, then those that are copied.
    const int heads = a.x[0].heads + a.x[1].heads, teams = kRotaryThreads / places > 0 ? kRotaryThreads / places : 1;
    const int step = kRotaryThreads / teams;   // threads of a team
    const int team = threadIdx.x / step;
    if (team >= teams) return;
    for (int i = team; i < rows * heads; i += teams) {
        const int r = i / heads, head = i % heads;
        const bool second = head >= a.x[0].heads;
        const RotaryRows& x = a.x[second];
        const int h = second ? head - a.x[0].heads : head;
        if (__ldg(a.positions + row0 + r) < 0) continue;
        const T* in = static_cast<const T*>(x.in.p) + (row0 + r) * x.in.row + h * x.in.head;
        T* out = static_cast<T*>(x.out.p) + (row0 + r) * x.out.row + h * x.out.head;
        [[maybe_unused]] const int64_t in_bytes = ((a.rows - 1) * x.in.row + (x.heads - 1) * x.in.head + a.dim) * (int64_t)sizeof(T);
        [[maybe_unused]] const int64_t out_bytes = ((a.rows - 1) * x.out.row + (x.heads - 1) * x.out.head + a.dim) * (int64_t)sizeof(T);
        for (int place = threadIdx.x % step; place < places; place += step) {
            const float2* by = s_by + r * half;
            if (place >= turned) {
                const int at = a.part + (place - turned) * PER;
                if (in == out || !GEMM_DBG_OK(in + at, x.in.p, in_bytes, PER * sizeof(T)) || !GEMM_DBG_OK(out + at, x.out.p, out_bytes, PER * sizeof(T))) continue;
                Piece<T, PER> e;
                e.load(in + at);
                e.store(out + at);
            } else if constexpr (INTERLEAVED && PER > 1) {
                const int at = place * PER;
                if (!GEMM_DBG_OK(in + at, x.in.p, in_bytes, PER * sizeof(T)) || !GEMM_DBG_OK(out + at, x.out.p, out_bytes, PER * sizeof(T))) continue;
                Piece<T, PER> e;
                e.load(in + at);
#pragma unroll
                for (int j = 0; j < PER; j += 2) {
                    const float2 w = by[at / 2 + j / 2];
                    const float u = e.v[j], v = e.v[j + 1];
                    e.v[j] = u * w.x - v * w.y;
                    e.v[j + 1] = v * w.x + u * w.y;
                }
                e.store(out + at);
            } else {
                const int at = place * PER * (INTERLEAVED ? 2 : 1), other = at + (INTERLEAVED ? 1 : half);
                if (!GEMM_DBG_OK(in + at, x.in.p, in_bytes, PER * sizeof(T)) || !GEMM_DBG_OK(in + other, x.in.p, in_bytes, PER * sizeof(T)) ||
                    !GEMM_DBG_OK(out + at, x.out.p, out_bytes, PER * sizeof(T)) || !GEMM_DBG_OK(out + other, x.out.p, out_bytes, PER * sizeof(T)))
                    continue;
                Piece<T, PER> e, f;
                e.load(in + at);
                f.load(in + other);
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    const float2 w = by[place * PER + j];
                    const float u = e.v[j], v = f.v[j];
                    e.v[j] = u * w.x - v * w.y;
                    f.v[j] = v * w.x + u * w.y;
                }
                e.store(out + at);
                f.store(out + other);
            }
        }
    }
}

template <typename T, int PER, bool INTERLEAVED>
cudaError_t rotate(const RotaryArgs& a, bool inverse, int num_sms, cudaStream_t stream) {
    const int turned = INTERLEAVED && PER > 1 ? a.part / PER : a.part / 2 / PER, places = turned + (a.dim - a.part) / PER;
    const int64_t each = a.rows / (8 * num_sms);
    const int rows = (int)(each < 1 ? 1 : each > 4 ? 4 : each);
    rotary_kernel<T, PER, INTERLEAVED><<<(unsigned)((a.rows + rows - 1) / rows), kRotaryThreads, rows * (a.part / 2) * sizeof(float2), stream>>>(
        a, rows, inverse, turned, places);
    return cudaGetLastError();
}

template <typename T>
cudaError_t rotate(const RotaryArgs& a, bool interleaved, bool inverse, int num_sms, cudaStream_t stream) {
    constexpr int kPer = 16 / sizeof(T);
    auto by16 = [](const KvRows& r) {
        return (reinterpret_cast<uintptr_t>(r.p) & 15u) == 0 && r.row * sizeof(T) % 16 == 0 && r.head * sizeof(T) % 16 == 0;
    };
    bool vec = a.part % (interleaved ? kPer : 2 * kPer) == 0 && a.dim % kPer == 0;
    for (const RotaryRows& x : a.x) vec = vec && (x.heads == 0 || (by16(x.in) && by16(x.out)));
    if (vec) return interleaved ? rotate<T, kPer, true>(a, inverse, num_sms, stream) : rotate<T, kPer, false>(a, inverse, num_sms, stream);
    return interleaved ? rotate<T, 1, true>(a, inverse, num_sms, stream) : rotate<T, 1, false>(a, inverse, num_sms, stream);
}

}  // namespace

LIBGEMM_DEBUG_READER(sequences_debug_flags)

cudaError_t launch_step_plan(const StepPlan& p, unsigned* err, int* launches, cudaStream_t stream) {
    const unsigned threads = p.sequences <= 256 ? 256 : kScanThreads;
    plan_scan_kernel<<<1, threads, 0, stream>>>(p, err);
    cudaError_t e = cudaGetLastError();
    *launches = 1;
    if (e != cudaSuccess || p.tokens == 0) return e;
    const int64_t units = p.tokens / kFillRows + p.sequences + 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((units + kFillThreads / 32 - 1) / (kFillThreads / 32)));
    cfg.blockDim = dim3(kFillThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = kUsePdl;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, plan_fill_kernel, p);
    *launches = 2;
    return e;
}

cudaError_t launch_rotary(const RotaryArgs& a, ElemType type, bool interleaved, bool inverse, int num_sms, cudaStream_t stream) {
    if (type == ElemType::kF32) return rotate<float>(a, interleaved, inverse, num_sms, stream);
    if (type == ElemType::kBF16) return rotate<__nv_bfloat16>(a, interleaved, inverse, num_sms, stream);
    return rotate<__half>(a, interleaved, inverse, num_sms, stream);
}

}  // namespace libgemm
