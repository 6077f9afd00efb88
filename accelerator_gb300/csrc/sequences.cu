// sequences.cu -- what a batch of sequences needs around a paged cache: the plan
// of a step (row offsets, pages, positions, slots) and rotary positions.
#include "kernels.h"
#include "lowbit.cuh"

namespace libgemm {
namespace {

// ---- the plan ------------------------------------------------------------------
// Sums over the sequences (rows, pages), a thread a sequence, give what is one
// number a sequence; then a warp takes 256 rows of a sequence, whose positions and
// slots follow from its first row, its length and its place on the stack alone: the
// new pages' numbers come off the stack, not out of the table, which the same lanes
// write.  For up to 1024 sequences every block makes the sums itself, in shared
// memory, and it is one launch; beyond that, or where lengths are written in place,
// one block makes them and a second launch reads them.  Latency bounds it: a plan of 64
// sequences takes 4.6 us of the GPU in one launch and 4.1 and 4.3 in two, one of 1000
// sequences of up to 512 rows 11.6 (3.1 MB of positions and slots written).  Recorded
// one after another, one launch and two (with lengths in place): 64 sequences of one row
// 2.8 and 3.1 us, 512 of up to 64 rows 4.5 and 7.2, 1000 of one row 5.6 and 6.7, 1024 5.8
// and 6.9; in two launches 1025 take 11.0, as the sums go through two rounds, 2000 11.2.
constexpr int kScanThreads = 1024, kFillThreads = 256, kFillRows = 256, kOneLaunch = 1024;

__device__ __forceinline__ int pages_of(int64_t tokens, const StepPlan& p) {   // columns of the table, which is all that are held
    const int64_t n = (tokens + (1 << p.page_log2) - 1) >> p.page_log2;
    return (int)(n < p.width ? n : p.width);
}

// The sums, by one block: put(b, start, first, height, after) of every sequence,
// and of b = sequences start and height alone.  True if a number is out of range.
template <typename F>
__device__ __forceinline__ bool plan_sums(const StepPlan& p, F put) {
    __shared__ int64_t s_rows[32], s_pages[32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    const int top = *p.available;
    const int height = top < 0 ? 0 : top > p.capacity ? (int)p.capacity : top;
    bool bad = height != top;
    auto left = [&](int64_t taken) { return (int)(height - taken > INT32_MIN ? height - taken : INT32_MIN); };
    int64_t rows0 = 0, pages0 = 0;   // of the sequences before this round's
    for (int64_t b0 = 0; b0 < p.sequences; b0 += blockDim.x) {
        const int64_t b = b0 + threadIdx.x;
        const bool in = b < p.sequences && GEMM_DBG_OK(p.lengths + b, p.lengths, p.sequences * 4, 4);
        const int length = in ? p.lengths[b] : 0, count = in ? __ldg(p.counts + b) : 0;
        const int held = max(length, 0);
        int added = max(count, 0);
        int64_t after = (int64_t)held + added, need = pages_of(after, p) - pages_of(held, p);
        bad |= length < 0 || count < 0 || (added > 0 && (after > p.width << p.page_log2 || after > INT32_MAX));
        int64_t rows, pages, rows_all, pages_all;   // sums up to this thread's sequence, and of all
        auto sum = [&] {
            rows = added, pages = need;
            for (int i = 1; i < 32; i *= 2) {
                const int64_t r = __shfl_up_sync(0xFFFFFFFFu, rows, i), g = __shfl_up_sync(0xFFFFFFFFu, pages, i);
                if (lane >= i) rows += r, pages += g;
            }
            __syncthreads();   // the last sums have been read
            if (lane == 31) s_rows[warp] = rows, s_pages[warp] = pages;
            __syncthreads();
            rows_all = pages_all = 0;
            for (int w = 0; w < warps; ++w) {
                if (w == warp) rows += rows_all, pages += pages_all;
                rows_all += s_rows[w], pages_all += s_pages[w];
            }
        };
        sum();
        if (rows0 + rows_all > p.tokens) {   // (all threads or none) a sequence gets what the rows have room for, and pages for that
            bad = true;
            const int64_t room = p.tokens - rows0 - (rows - added);
            if (added > room) added = room > 0 ? (int)room : 0;
            after = (int64_t)held + added, need = pages_of(after, p) - pages_of(held, p);
            sum();
        }
        if (in) {
            bad |= pages0 + pages > height && need > 0;
            put(b, (int)(rows0 + rows - added), held, left(pages0 + pages - need), (int)(after < INT32_MAX ? after : INT32_MAX));
        }
        rows0 += rows_all, pages0 += pages_all;
    }
    __syncthreads();   // every thread has read `available`, which may be `left`
    if (threadIdx.x == 0) put(p.sequences, (int)rows0, 0, left(pages0), 0);
    return bad;
}

__device__ __forceinline__ void plan_put(const StepPlan& p, int64_t b, int start, int first, int height, int after) {
    if (!GEMM_DBG_OK(p.starts + b, p.starts, (p.sequences + 1) * 4, 4) || !GEMM_DBG_OK(p.heights + b, p.heights, (p.sequences + 1) * 4, 4)) return;
    p.starts[b] = start;
    p.heights[b] = height;
    if (b == p.sequences) *p.left = max(height, 0);
    else if (GEMM_DBG_OK(p.first + b, p.first, p.sequences * 4, 4) && GEMM_DBG_OK(p.after + b, p.after, p.sequences * 4, 4)) p.first[b] = first, p.after[b] = after;
}

// Unit u of the rows, by one warp: sequence b's are units floor(starts[b] / 256) + b
// + j, and those past the last sequence's the same of one more.
template <typename S, typename F, typename H>
__device__ __forceinline__ void plan_fill(const StepPlan& p, int64_t u, S start, F first_of, H height_of) {
    const int n = (int)p.sequences;
    const int b = last_not_above(n + 1, u, u, [&](int i) { return (int64_t)start(i) / kFillRows + i; });
    const int64_t row0 = start(b), end = b < n ? start(b + 1) : p.tokens;
    const int64_t begin = row0 + (u - row0 / kFillRows - b) * kFillRows;
    if (begin >= end) return;
    const int first = b < n ? first_of(b) : 0, height = b < n ? height_of(b) : 0, held = pages_of(first, p);
    int32_t* table = p.table + (int64_t)b * p.width;
    for (int64_t row = begin + threadIdx.x % 32; row < min(end, begin + kFillRows); row += 32) {
        int position = -1;
        int64_t slot = -1;
        if (b < n) {
            const int64_t at = first + (row - row0);
            position = at <= INT32_MAX ? (int)at : -1;
            const int64_t column = at >> p.page_log2;
            const int in = (int)(at & ((1 << p.page_log2) - 1));
            if (column < p.width && position >= 0 && GEMM_DBG_OK(table + column, p.table, p.sequences * p.width * 4, 4)) {
                int page;
                if (column < held) {
                    page = table[column];
                } else {   // new, off the stack; its first token writes the table
                    const int64_t from = height - 1 - (column - held);
                    page = from >= 0 && GEMM_DBG_OK(p.free + from, p.free, p.capacity * 4, 4) ? __ldg(p.free + from) : -1;
                    if (in == 0) table[column] = page;
                }
                if (page >= 0) slot = ((int64_t)page << p.page_log2) + in;
            }
        }
        if (!GEMM_DBG_OK(p.positions + row, p.positions, p.tokens * 4, 4) || !GEMM_DBG_OK(p.slots + row, p.slots, p.tokens * 8, 8)) continue;
        p.positions[row] = position;
        p.slots[row] = slot;
    }
}

__global__ void __launch_bounds__(kFillThreads) plan_kernel(StepPlan p, unsigned* err) {
    __shared__ int s_start[kOneLaunch + 1], s_first[kOneLaunch], s_height[kOneLaunch + 1];
    const bool bad = plan_sums(p, [&](int64_t b, int start, int first, int height, int after) {
        s_start[b] = start, s_height[b] = height;
        if (b < p.sequences) s_first[b] = first;
        if (blockIdx.x == 0) plan_put(p, b, start, first, height, after);
    });
    if (bad && blockIdx.x == 0) atomicOr(err, kErrIndex);
    __syncthreads();
    const int64_t u = (int64_t)blockIdx.x * (kFillThreads / 32) + threadIdx.x / 32;
    plan_fill(p, u, [&](int b) { return s_start[b]; }, [&](int b) { return s_first[b]; }, [&](int b) { return s_height[b]; });
}

__global__ void __launch_bounds__(kScanThreads) plan_scan_kernel(StepPlan p, unsigned* err) {
    grid_launch_dependents();
    const bool bad = plan_sums(p, [&](int64_t b, int start, int first, int height, int after) { plan_put(p, b, start, first, height, after); });
    if (bad) atomicOr(err, kErrIndex);
}

__global__ void __launch_bounds__(kFillThreads) plan_fill_kernel(StepPlan p) {
    grid_dependency_wait();
    const int64_t u = (int64_t)blockIdx.x * (kFillThreads / 32) + threadIdx.x / 32;
    plan_fill(p, u, [&](int b) { return p.starts[b]; }, [&](int b) { return p.first[b]; }, [&](int b) { return p.heights[b]; });
}

// ---- rotary positions ------------------------------------------------------------
// A block has some rows with all heads of both operands.  Its threads first make
// the rows' sines and cosines, one a pair, in shared memory: the angle is
// position * turns mod 2^64 in fractions of a turn, one integer product without any
// loss.  The nearest quarter turn is taken off in integers, and what is left, an eighth
// of a turn at most, is rounded to binary32 once, all 64 bits of it: a sine next to one
// of its zeros keeps its relative error.  Then each thread has one place of a head -- PER elements of either half, or PER
// neighbours -- and goes through heads and rows, kAhead of them loaded before the
// first is used.  11000 rows of 40 heads of 128, bfloat16: 39 us, 225 MB at 5.7
// TB/s, 85 % of the measured copy rate; the L1 pipe is at 83 %.  Before the pairs were
// packed, one place ahead took 41.6 us, two 42.9 and four 45.9 (74 registers), and two
// the least for few rows.  A row a team with its sines kept in registers takes 39.5
// and, for 2000 rows of 24 heads that turn 32 of 128 dimensions, 10.7 where this takes 8.5.
// (All of these with 32 bits of the angle; with 64, recorded: 40.1 -> 40.6 us, 6.2 -> 6.5
// for that part.)  9700 rows of 20 heads of 64, 50 MB: 13.8 us out of a cold L2, where the
// copy rate would give 7.4: the SMs are at work for 69 % of it, the rest is the launch's
// beginning and end, and then issue 0.58 instructions a cycle and scheduler.
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
    uint4 v;
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (PER == 1) v.x = __float_as_uint(as_float(*p));
        else v = *reinterpret_cast<const uint4*>(p);
    }
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (PER == 1) *p = from_float<T>(__uint_as_float(v.x));
        else *reinterpret_cast<uint4*>(p) = v;
    }
    __device__ __forceinline__ void get(float (&f)[PER]) const {
        if constexpr (PER == 1) f[0] = __uint_as_float(v.x);
        else {
            const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
            for (int i = 0; i < PER; ++i) f[i] = as_float(e[i]);
        }
    }
    __device__ __forceinline__ void put(const float (&f)[PER]) {
        if constexpr (PER == 1) v.x = __float_as_uint(f[0]);
        else if constexpr (PER == 4) v = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
        else v = make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7]));
    }
};

constexpr int kAhead = 2;
// Rows of a block: the rule at the launch would take more for very few heads, whose
// threads then have nothing to turn.  100000 rows of 64 dimensions: 16 + 4 heads 91 us
// (5.6 TB/s), 8 + 2 59 (4.3), 4 + 1 46, 2 + 1 42, 1 + 1 40 (1.3).
constexpr int kMaxRows = 8;

template <typename T, int PER, bool INTERLEAVED>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const RotaryArgs a, int rows_each, bool inverse, int turned, int places) {
    extern __shared__ __align__(16) float s_by[];   // cosines, then sines: [rows][pairs] each
    __shared__ bool s_off[kMaxRows];                // rows that stay as they are
    constexpr bool kTwo = !INTERLEAVED || PER == 1; // a turned place is two pieces
    constexpr int kPairs = kTwo ? PER : PER / 2;    // of a turned place
    const int half = a.part / 2;
    const int64_t row0 = (int64_t)blockIdx.x * rows_each;
    const int rows = (int)(a.rows - row0 < rows_each ? a.rows - row0 : rows_each);
    const float *s_cos = s_by, *s_sin = s_by + rows_each * half;
    // Places of a head: `turned` that turn, then those that are copied.  A team of
    // threads has all places of one head, in turns if it has fewer threads.
    const int heads = a.x[0].heads + a.x[1].heads, step = places < kRotaryThreads ? places : kRotaryThreads, teams = kRotaryThreads / step;
    const int team = threadIdx.x / step;

    struct Item {
        Piece<T, PER> e, f;
        T* out;
        int r, pair;                 // pair < 0: copied
        bool live;
    };
    auto load = [&](Item& it, int r, int head, int place) {
        const bool second = head >= a.x[0].heads;
        const RotaryRows& x = a.x[second];
        const int h = second ? head - a.x[0].heads : head;
        const bool copied = place >= turned;
        const int at = copied ? a.part + (place - turned) * PER : place * PER * (INTERLEAVED && PER == 1 ? 2 : 1);
        const T* in = static_cast<const T*>(x.in.p) + (row0 + r) * x.in.row + h * x.in.head + at;
        it.out = static_cast<T*>(x.out.p) + (row0 + r) * x.out.row + h * x.out.head + at;
        it.r = r;
        it.pair = copied ? -1 : place * kPairs;
        [[maybe_unused]] const int64_t in_bytes = ((a.rows - 1) * x.in.row + (x.heads - 1) * x.in.head + a.dim) * (int64_t)sizeof(T);
        [[maybe_unused]] const int64_t out_bytes = ((a.rows - 1) * x.out.row + (x.heads - 1) * x.out.head + a.dim) * (int64_t)sizeof(T);
        const int other = INTERLEAVED ? 1 : half;
        it.live = !(copied && in == it.out) && GEMM_DBG_OK(in, x.in.p, in_bytes, PER * sizeof(T)) && GEMM_DBG_OK(it.out, x.out.p, out_bytes, PER * sizeof(T));
        if (kTwo && it.live && !copied)
            it.live = GEMM_DBG_OK(in + other, x.in.p, in_bytes, PER * sizeof(T)) && GEMM_DBG_OK(it.out + other, x.out.p, out_bytes, PER * sizeof(T));
        if (!it.live) return;
        it.e.load(in);
        if (kTwo && !copied) it.f.load(in + other);
    };
    auto finish = [&](Item& it) {
        if (!it.live || s_off[it.r]) return;
        if (it.pair >= 0) {
            float u[kPairs], v[kPairs], c[kPairs], n[kPairs];   // the pairs, cosines and sines
            if constexpr (kTwo) {
                it.e.get(u);
                it.f.get(v);
            } else {
                float both[PER];
                it.e.get(both);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) u[j] = both[2 * j], v[j] = both[2 * j + 1];
            }
            const int at = it.r * half + it.pair;
            if constexpr (kPairs == 1) {
                c[0] = s_cos[at], n[0] = s_sin[at];
                const float x = u[0] * c[0] - v[0] * n[0];
                v[0] = v[0] * c[0] + u[0] * n[0];
                u[0] = x;
            } else {
#pragma unroll
                for (int j = 0; j < kPairs; j += 2) {
                    const float2 c2 = *reinterpret_cast<const float2*>(s_cos + at + j), n2 = *reinterpret_cast<const float2*>(s_sin + at + j);
                    const float2 u2 = make_float2(u[j], u[j + 1]), v2 = make_float2(v[j], v[j + 1]), m2 = make_float2(-n2.x, -n2.y);
                    const float2 x = __ffma2_rn(u2, c2, __fmul2_rn(v2, m2)), y = __ffma2_rn(v2, c2, __fmul2_rn(u2, n2));
                    u[j] = x.x, u[j + 1] = x.y, v[j] = y.x, v[j + 1] = y.y;
                }
            }
            if constexpr (kTwo) {
                it.e.put(u);
                it.f.put(v);
                it.f.store(it.out + (INTERLEAVED ? 1 : half));
            } else {
                float both[PER];
#pragma unroll
                for (int j = 0; j < kPairs; ++j) both[2 * j] = u[j], both[2 * j + 1] = v[j];
                it.e.put(both);
            }
        }
        it.e.store(it.out);
    };

    int r = 0, head = team, place = team < teams ? threadIdx.x % step : places;
    auto settle = [&] {   // head numbers past the last go on in the next row
        while (r < rows && head >= heads) head -= heads, ++r;
    };
    auto next = [&](Item (&item)[kAhead]) {   // false if there was none
        if (place >= places) return false;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            item[i].live = false;
            if (r < rows) {
                load(item[i], r, head, place);
                head += teams;
                settle();
            }
        }
        if (r >= rows) {
            r = 0, head = team, place += step;
            settle();
        }
        return true;
    };
    settle();
    if (r >= rows) place = places;   // a team past the last head of the last row
    Item item[kAhead];
    bool some = next(item);   // under way while the sines are made
    for (int i = threadIdx.x; i < rows * half; i += kRotaryThreads) {
        const int at = i / half, pair = i % half;
        const int position = __ldg(a.positions + row0 + at);
        const uint64_t turn = (uint64_t)(uint32_t)position * __ldg(a.turns + pair);
        const uint64_t quarters = (turn + (1ull << 61)) >> 62;   // to the nearest, modulo 4
        float n, c;
        sincospif(__ll2float_rn((int64_t)(turn - (quarters << 62))) * 1.0842021724855044e-19f, &n, &c);   // 2^-63
        if (quarters & 1) {
            const float x = n;
            n = c, c = -x;
        }
        if (quarters & 2) n = -n, c = -c;
        s_by[i] = c * a.magnitude;
        s_by[rows_each * half + i] = (inverse ? -n : n) * a.magnitude;
    }
    if (threadIdx.x < rows) s_off[threadIdx.x] = __ldg(a.positions + row0 + threadIdx.x) < 0;
    __syncthreads();
    for (; some; some = next(item))
#pragma unroll
        for (int i = 0; i < kAhead; ++i) finish(item[i]);
}

template <typename T, int PER, bool INTERLEAVED>
cudaError_t rotate(const RotaryArgs& a, bool inverse, int num_sms, cudaStream_t stream) {
    const int turned = INTERLEAVED && PER > 1 ? a.part / PER : a.part / 2 / PER, places = turned + (a.dim - a.part) / PER;
    // About four places a thread, unless that leaves SMs without a block.
    const int64_t most = a.rows / (4 * num_sms), want = 4 * kRotaryThreads / ((int64_t)(a.x[0].heads + a.x[1].heads) * places);
    const int64_t each = most < want ? most : want;
    const int rows = (int)(each < 1 ? 1 : each > kMaxRows ? kMaxRows : each);
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
    // Pieces of 16 bytes where all of them fit, one element else.  11000 rows of 20 heads
    // of bfloat16, recorded: halves of 80 of 80 dimensions 14 us, 40 of 80 60 (neighbours:
    // 15), 32 of 96 19 and 24 of 96 72; 40 heads of 128 41, one element off 16 bytes 127.
    bool vec = a.part % (interleaved ? kPer : 2 * kPer) == 0 && a.dim % kPer == 0;
    for (const RotaryRows& x : a.x) vec = vec && (x.heads == 0 || (by16(x.in) && by16(x.out)));
    if (vec) return interleaved ? rotate<T, kPer, true>(a, inverse, num_sms, stream) : rotate<T, kPer, false>(a, inverse, num_sms, stream);
    return interleaved ? rotate<T, 1, true>(a, inverse, num_sms, stream) : rotate<T, 1, false>(a, inverse, num_sms, stream);
}

}  // namespace

LIBGEMM_DEBUG_READER(sequences_debug_flags)

cudaError_t launch_step_plan(const StepPlan& p, unsigned* err, int* launches, cudaStream_t stream) {
    const int64_t units = p.tokens / kFillRows + p.sequences + 1;
    const unsigned blocks = (unsigned)((units + kFillThreads / 32 - 1) / (kFillThreads / 32));
    *launches = 1;
    if (p.sequences <= kOneLaunch && p.after != p.lengths && p.left != p.available) {
        plan_kernel<<<blocks, kFillThreads, 0, stream>>>(p, err);
        return cudaGetLastError();
    }
    plan_scan_kernel<<<1, p.sequences <= 256 ? 256 : kScanThreads, 0, stream>>>(p, err);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.tokens == 0) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
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
