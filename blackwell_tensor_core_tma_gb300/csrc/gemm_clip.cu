// The Euclidean norm of many tensors together, and the tensors scaled to a largest norm (gemm_clip_run in
// include/gb300gemm.h):
//
//   norm = sqrt(sum g^2),  c = g * min(1, limit / norm)
//
// Two kernels over the same rows of ROW bytes, each CTA with a range of consecutive ones.  The first leaves each CTA's sum of
// squares; in the second every CTA adds those up, in the same order, so that no counter stands between them, and scales its
// range from its end: what the first kernel read last is still in L2.  Few rows are left to one cluster, which does both at
// once.  A list that is longer than a launch's parameters goes through several of the first kernel, whose CTAs add to the sums
// that those before them left, and as many of the second.
//
// Sums: a thread squares and adds the values of a step (16 or 32 of them) in fp32 and adds that sum to a pair of fp32 numbers
// whose sum carries twice fp32's digits.  Where a step's largest magnitude takes squares or sums past fp32's ends it is
// scaled by a power of two first and its sum kept in 64 bits.  (In 64 bits throughout, the sums of a CTA's threads, the root
// and the quotient alone took 5 us: the unit has two lanes per SM and clock.)
#include <algorithm>
#include <type_traits>

#include "gemm_rows.cuh"

namespace gb300 {
namespace {

using namespace rows;

constexpr int THREADS = 256;
constexpr int ROW = THREADS * 16;                          // bytes: a 16-byte piece for each thread
constexpr int STEP = 4;                                    // rows that a CTA takes at a time, of one tensor

// ------------------------------------------------------------------------------------------- the list

struct Entry {
    const uint8_t *g;
    uint8_t *c;
    int64_t n;
    uint32_t first;          // its first row
    int16_t type;
    int16_t apart;           // c is not a multiple of 16 bytes from g: written element by element
};
// What a CTA leaves: its sum of squares is high + low + rest
struct Part {
    float high, low;
    double rest;             // of what fp32 does not hold
};
constexpr int MAX_PARTS = GEMM_CLIP_WORKSPACE / (int)sizeof(Part);
// The tensors of one launch, by value: a captured graph keeps them.  start[b]: the tensor of CTA b's first row.  (Looked up
// by halving in the launch's parameters, it costs a cache miss per step: 500 tensors of 1000 elements took 20 us, not 12.)
template <int N, int CTAS = MAX_PARTS>
struct Table {
    int count;
    uint32_t rows;
    bool copies;             // some c is not its g
    uint16_t start[CTAS];
    Entry e[N];
};

// A CTA's rows [begin, end)
struct Range {
    uint32_t begin, end;
};
__host__ __device__ __forceinline__ Range range_of(uint32_t rows, uint32_t cta, uint32_t ctas) {
    return {(uint32_t)((uint64_t)rows * cta / ctas), (uint32_t)((uint64_t)rows * (cta + 1) / ctas)};
}

__device__ __forceinline__ float load_one(const uint8_t *g, int type, int64_t i) {
    if (type == GEMM_F32) return reinterpret_cast<const float *>(g)[i];
    if (type == GEMM_BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(g)[i]);
    return __half2float(reinterpret_cast<const __half *>(g)[i]);
}
__device__ __forceinline__ void store_one(uint8_t *c, int type, int64_t i, float v) {
    if (type == GEMM_F32) reinterpret_cast<float *>(c)[i] = v;
    else if (type == GEMM_BF16) reinterpret_cast<__nv_bfloat16 *>(c)[i] = __float2bfloat16_rn(v);
    else reinterpret_cast<__half *>(c)[i] = __float2half_rn(v);
}

// A tensor's elements before its first 16-byte boundary, its whole pieces and the elements behind them
struct Span {
    int head, tail;
    int64_t pieces;
    __device__ __forceinline__ Span(const Entry &e) {
        const int size = e.type == GEMM_F32 ? 4 : 2, per = 16 / size;
        head = (int)((16 - (reinterpret_cast<uintptr_t>(e.g) & 15)) & 15) / size;
        if (head > e.n) head = (int)e.n;
        pieces = (e.n - head) / per;
        tail = (int)(e.n - head - pieces * per);
    }
};

// What L2 does with lines that a kernel is through with: leave in their turn, or first
__device__ __forceinline__ uint64_t in_turn() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ uint64_t first_out() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
// The pieces of a step: a thread's are thread, thread + THREADS, ..., zeros past the step's own.  While a step's are worked
// on, those of the next one are on their way into the same registers.
struct Pieces {
    uint4 q[STEP];
    uint64_t policy;
    __device__ __forceinline__ void load(int i, const uint4 *g, int left, int thread) {
        const uint4 *from = g + (i * THREADS + thread);
        q[i] = make_uint4(0, 0, 0, 0);
        if (i * THREADS + thread < left)
            asm volatile("ld.global.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
                         : "=r"(q[i].x), "=r"(q[i].y), "=r"(q[i].z), "=r"(q[i].w)
                         : "l"(from), "l"(policy)
                         : "memory");
    }
    __device__ __forceinline__ void store(uint4 *to, const uint4 &v) const {
        asm volatile("st.global.L2::cache_hint.v4.u32 [%0], {%1, %2, %3, %4}, %5;" ::"l"(to), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w),
                     "l"(policy)
                     : "memory");
    }
};

// A walk over a range's rows, up to STEP of one tensor at a time
template <typename T>
struct Walk {
    const T &t;
    int i;                   // the step's tensor
    uint32_t row, rows;      // the step: rows of the list [row, row + rows)
    const uint4 *g;          // its pieces
    int left;                // how many
    __device__ __forceinline__ Walk(const T &table, int start) : t(table), i(start), row(0), rows(0), g(nullptr), left(0) {}
    __device__ __forceinline__ void up(uint32_t from, const Range &r) {            // the step that begins at `from`
        while (i + 1 < t.count && t.e[i + 1].first <= from) ++i;
        row = from;
        const uint32_t end = i + 1 < t.count ? min(t.e[i + 1].first, r.end) : r.end;
        rows = min((uint32_t)STEP, end - from);
        place();
    }
    __device__ __forceinline__ void down(uint32_t to, const Range &r) {            // the step that ends at `to`
        while (i + 1 < t.count && t.e[i + 1].first < to) ++i;
        while (t.e[i].first >= to) --i;
        const uint32_t begin = max(t.e[i].first, r.begin);
        rows = min((uint32_t)STEP, to - begin);
        row = to - rows;
        place();
    }
    __device__ __forceinline__ void none() { left = 0; }

private:
    __device__ __forceinline__ void place() {
        const Entry &e = t.e[i];
        const Span s(e);
        const int64_t at = (int64_t)(row - e.first) * THREADS;
        g = reinterpret_cast<const uint4 *>(e.g + s.head * (e.type == GEMM_F32 ? 4 : 2)) + at;
        left = (int)max((int64_t)0, min(s.pieces - at, (int64_t)(rows * THREADS)));
    }
};

// ------------------------------------------------------------------------------------------- sums

// not zero, by its bits: a comparison in 64 bits takes the slow unit too
__device__ __forceinline__ bool any_bits(double v) { return (__double2hiint(v) | __double2loint(v)) != 0; }

// high + low, low what high's rounding left; and what fp32 does not hold
struct Sum {
    float high = 0.f, low = 0.f;
    double rest = 0.0;
    __device__ __forceinline__ void add(float v) {
        const float s = high + v, z = s - high;
        low += (high - (s - z)) + (v - z);
        high = s;
    }
    __device__ __forceinline__ void add(const Part &p) {
        add(p.high);
        low += p.low;
        if (any_bits(p.rest)) rest += p.rest;
    }
};
__device__ __forceinline__ Sum warp_sum(Sum s) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        const float h = __shfl_xor_sync(0xFFFFFFFFu, s.high, o), l = __shfl_xor_sync(0xFFFFFFFFu, s.low, o);
        // the same in both lanes of a pair
        const float a = fmaxf(s.high, h), b = fminf(s.high, h), t = a + b;
        s.low = (s.low + l) + (b - (t - a));
        s.high = s.high != s.high || h != h ? s.high + h : t;
    }
    if (__any_sync(0xFFFFFFFFu, any_bits(s.rest))) {
#pragma unroll
        for (int o = 16; o > 0; o /= 2) s.rest += __shfl_xor_sync(0xFFFFFFFFu, s.rest, o);
    }
    return s;
}
// Over a CTA, in the same order every time; valid in all threads
__device__ __forceinline__ Sum block_sum(const Sum &v) {
    __shared__ Part warps[THREADS / 32];
    const Sum w = warp_sum(v);
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x / 32] = Part{w.high, w.low, w.rest};
    __syncthreads();
    Sum s;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) s.add(warps[i]);
    return s;
}

// f(pair of values) for a piece
template <int TYPE, typename F>
__device__ __forceinline__ void pairs(const uint4 &q, F f) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    if constexpr (TYPE == GEMM_F32) {
        f(make_float2(__uint_as_float(w[0]), __uint_as_float(w[1])));
        f(make_float2(__uint_as_float(w[2]), __uint_as_float(w[3])));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (TYPE == GEMM_BF16) f(make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)));
            else f(__half22float2(*reinterpret_cast<const __half2 *>(&w[i])));
        }
    }
}
// The largest magnitude of a thread's values, NaN left out
template <int TYPE>
__device__ __forceinline__ float largest(const Pieces &p) {
    if constexpr (TYPE == GEMM_F32) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < STEP; ++i) pairs<TYPE>(p.q[i], [&](float2 v) { m = fmaxf(m, fmaxf(fabsf(v.x), fabsf(v.y))); });
        return m;
    } else {
        using T2 = typename std::conditional<TYPE == GEMM_BF16, __nv_bfloat162, __half2>::type;
        const uint32_t zero = 0;
        T2 m = *reinterpret_cast<const T2 *>(&zero);
#pragma unroll
        for (int i = 0; i < STEP; ++i) {
            const uint32_t w[4] = {p.q[i].x, p.q[i].y, p.q[i].z, p.q[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) m = __hmax2(m, __habs2(*reinterpret_cast<const T2 *>(&w[k])));
        }
        return fmaxf(fabsf((float)m.x), fabsf((float)m.y));
    }
}

// A step's squares.  With every magnitude at most 2^40, and the largest at least 2^-56, neither squares nor the sums of 2^43
// of them leave fp32's range, and what squares below its normal numbers lose does not count beside the largest.
template <int TYPE, typename W>
__device__ __forceinline__ void add_squares(Pieces &p, const W &next, int thread, Sum &sum) {
    float2 s[2] = {};
#pragma unroll
    for (int i = 0; i < STEP; ++i) {
        int k = 0;
        pairs<TYPE>(p.q[i], [&](float2 v) { s[k] = fma2(v, v, s[k]); k ^= 1; });
    }
    const float amax = largest<TYPE>(p);
    if (amax > 0x1p40f || (amax < 0x1p-56f && amax != 0.f)) {
        const float2 shift = both(amax > 1.f ? 0x1p-70f : 0x1p90f);
        s[0] = s[1] = both(0.f);
#pragma unroll
        for (int i = 0; i < STEP; ++i) {
            int k = 0;
            pairs<TYPE>(p.q[i], [&](float2 v) {
                v = mul2(v, shift);
                s[k] = fma2(v, v, s[k]);
                k ^= 1;
            });
        }
        sum.rest += (double)((s[0].x + s[0].y) + (s[1].x + s[1].y)) * (amax > 1.f ? 0x1p140 : 0x1p-180);
    } else {
        sum.add((s[0].x + s[0].y) + (s[1].x + s[1].y));
    }
#pragma unroll
    for (int i = 0; i < STEP; ++i) p.load(i, next.g, next.left, thread);
}
__device__ __forceinline__ void add_square(float v, Sum &sum) {
    const float a = fabsf(v);
    if (a <= 0x1p40f && a >= 0x1p-56f) sum.add(v * v);
    else if (v != 0.f) sum.rest += (double)v * (double)v;
}

// The squares of a range, of which the last `keep` rows are to stay in L2
template <typename T>
__device__ __forceinline__ void norm_rows(const T &t, const Range &r, int start, int thread, uint32_t keep, Sum &sum) {
    if (r.begin >= r.end) return;
    const uint64_t stay = in_turn(), leave = first_out();
    Walk<T> next(t, start);
    Pieces p;
    p.policy = r.end - r.begin > keep ? leave : stay;
    next.up(r.begin, r);
#pragma unroll
    for (int i = 0; i < STEP; ++i) p.load(i, next.g, next.left, thread);
    for (uint32_t row = r.begin; row < r.end;) {
        const Entry &e = t.e[next.i];
        const bool first = row == e.first;
        row += next.rows;
        if (row < r.end) next.up(row, r); else next.none();
        p.policy = r.end - row > keep ? leave : stay;
        if (e.type == GEMM_F32) add_squares<GEMM_F32>(p, next, thread, sum);
        else if (e.type == GEMM_BF16) add_squares<GEMM_BF16>(p, next, thread, sum);
        else add_squares<GEMM_F16>(p, next, thread, sum);
        if (first) {                                       // at most seven elements before and behind the pieces
            const Span s(e);
            if (thread < s.head) add_square(load_one(e.g, e.type, thread), sum);
            if (thread < s.tail) add_square(load_one(e.g, e.type, e.n - s.tail + thread), sum);
        }
    }
}

// limit / norm as a product of two: where it is below 2^-100, a power of two and the rest.  The rest comes first: it is below one,
// and where it takes a value below fp32's normal numbers the power leaves zero of that.
struct Factor {
    float rest, power;
    bool one;
    __device__ __forceinline__ float operator()(float v) const { return v * rest * power; }
};
// min(1, limit / norm); a norm that is not a number makes a factor that is none
__device__ __forceinline__ Factor factor_of(const Sum &s, float limit, float &norm) {
    if (!any_bits(s.rest) && s.high >= 0x1p-100f) {            // at least the largest square, and at most 2^125
        norm = sqrtf(s.high + s.low);
        if (norm <= limit) return {1.f, 1.f, true};
        const float ratio = limit / norm;
        if (ratio >= 0x1p-100f) return {ratio, 1.f, false};
        return {limit * 0x1p100f / norm, 0x1p-100f, false};
    }
    const double exact = sqrt((double)s.high + (double)s.low + s.rest), ratio = (double)limit / exact;
    norm = (float)exact;
    const bool one = exact <= (double)limit;
    const float power = ratio < 0x1p-100 ? 0x1p-100f : 1.f;
    return {one ? 1.f : (float)(ratio / (double)power), one ? 1.f : power, one};
}

// ------------------------------------------------------------------------------------------- results

template <int TYPE, typename W>
__device__ __forceinline__ void scale_pieces(Pieces &p, uint4 *to, int left, const W &next, int thread, const Factor &factor) {
    const float2 rest = make_float2(factor.rest, factor.rest), none = make_float2(-0.f, -0.f);      // x * rest + -0 is x * rest
#pragma unroll
    for (int i = 0; i < STEP; ++i) {
        float v[8];
        int n = 0;
        pairs<TYPE>(p.q[i], [&](float2 f) {
            f = fma2(f, rest, none);
            if (factor.power != 1.f) {
                f.x *= factor.power;
                f.y *= factor.power;
            }
            v[n++] = f.x;
            v[n++] = f.y;
        });
        uint4 q;
        if constexpr (TYPE == GEMM_F32)
            q = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        else if constexpr (TYPE == GEMM_BF16) q = pack8(static_cast<const __nv_bfloat16 *>(nullptr), v);
        else q = pack8(static_cast<const __half *>(nullptr), v);
        if (i * THREADS + thread < left) p.store(to + (i * THREADS + thread), q);
        p.load(i, next.g, next.left, thread);
    }
}

// A step's rows of a c that lies otherwise on its lines than g: element by element
__device__ __forceinline__ void scale_apart(const Entry &e, uint32_t row, uint32_t rows, int thread, const Factor &factor) {
    const Span s(e);
    const int per = e.type == GEMM_F32 ? 4 : 8;
    const int64_t at = (int64_t)row * THREADS, pieces = max((int64_t)0, min(s.pieces - at, (int64_t)(rows * THREADS)));
    const int64_t begin = s.head + at * per;
    for (int k = thread; k < pieces * per; k += THREADS)
        store_one(e.c, e.type, begin + k, factor(load_one(e.g, e.type, begin + k)));
}

// A range scaled, its last rows first; `leave`: what it reads and writes leaves L2 first
template <typename T>
__device__ __forceinline__ void scale_rows(const T &t, const Range &r, int start, int thread, bool leave, const Factor &factor) {
    if (r.begin >= r.end || (factor.one && !t.copies)) return;
    Walk<T> next(t, start);
    Pieces p;
    p.policy = leave ? first_out() : in_turn();
    auto down = [&](uint32_t to) {                         // nothing to load where nothing is written, or apart
        next.down(to, r);
        const Entry &e = t.e[next.i];
        if (!e.c || e.apart || (factor.one && e.c == e.g)) next.none();
    };
    down(r.end);
#pragma unroll
    for (int i = 0; i < STEP; ++i) p.load(i, next.g, next.left, thread);
    for (uint32_t row = r.end; row > r.begin;) {
        const Entry &e = t.e[next.i];
        const uint32_t rows = next.rows;
        const int left = next.left;
        uint4 *to = reinterpret_cast<uint4 *>(e.c + (reinterpret_cast<const uint8_t *>(next.g) - e.g));
        row = next.row;
        if (row > r.begin) down(row); else next.none();
        if (e.type == GEMM_F32) scale_pieces<GEMM_F32>(p, to, left, next, thread, factor);
        else if (e.type == GEMM_BF16) scale_pieces<GEMM_BF16>(p, to, left, next, thread, factor);
        else scale_pieces<GEMM_F16>(p, to, left, next, thread, factor);
        if (!e.c || (factor.one && e.c == e.g)) continue;
        if (e.apart) scale_apart(e, row - e.first, rows, thread, factor);
        if (row == e.first) {
            const Span s(e);
            if (thread < s.head) store_one(e.c, e.type, thread, factor(load_one(e.g, e.type, thread)));
            if (thread < s.tail) {
                const int64_t k = e.n - s.tail + thread;
                store_one(e.c, e.type, k, factor(load_one(e.g, e.type, k)));
            }
        }
    }
}

// ------------------------------------------------------------------------------------------- kernels

// Bound by memory, which the tensors pass three times.  CTAS_PER_SM of them run at once on an SM, and the grid is at most that
// many: no second wave.  1 billion fp32 values: 1.77 ms, 6750 GB/s over the three passes (a copy's rate); 100.7 million 190 us,
// 6370 GB/s; 40 million in 291 tensors of both types, copied, 62 us.  Steps of eight rows, four or six CTAs: within 3 %; loads
// past L1: the same.
constexpr int CTAS_PER_SM = 5;
template <int N>
__global__ void __launch_bounds__(THREADS, CTAS_PER_SM) clip_norm_kernel(const __grid_constant__ Table<N> t, Part *parts, int before, uint32_t keep) {
    const Range r = range_of(t.rows, blockIdx.x, gridDim.x);
    const int start = t.start[blockIdx.x];
    Sum sum;
    wait_for_previous();
    let_next_launch();
    norm_rows(t, r, start, threadIdx.x, keep, sum);
    sum = block_sum(sum);
    if (threadIdx.x == 0) {
        if ((int)blockIdx.x < before) sum.add(parts[blockIdx.x]);          // of the launches before this one
        parts[blockIdx.x] = Part{sum.high, sum.low, sum.rest};
    }
}

template <int N>
__global__ void __launch_bounds__(THREADS, CTAS_PER_SM)
    clip_scale_kernel(const __grid_constant__ Table<N> t, const Part *parts, int n, float limit, float *norm_out, bool leave) {
    const Range r = range_of(t.rows, blockIdx.x, gridDim.x);
    const int start = t.start[blockIdx.x];
    wait_for_previous();
    let_next_launch();
    Sum sum;
    for (int k = threadIdx.x; k < n; k += THREADS) sum.add(parts[k]);
    float norm;
    const Factor factor = factor_of(block_sum(sum), limit, norm);
    if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
    scale_rows(t, r, start, threadIdx.x, leave, factor);
}

// Few rows: one cluster does both, its CTAs' sums exchanged through shared memory.  A CTA has at most a row for each of its warps:
// a thread holds its pieces of all of them, read at once, and warp i's lanes the elements before and behind the pieces of the
// tensor that begins in row i.  Nothing is read twice: 20 011 values in 9 tensors 5.4 us.  (Without the barrier ahead of
// the exchange, which it needs, 5.0, and so 7.2 with the rows walked twice.)
constexpr int FEW_CTAS = 8, FEW_HELD = THREADS / 32;
constexpr uint32_t FEW_ROWS = FEW_CTAS * FEW_HELD;

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

template <int TYPE>
__device__ __forceinline__ void add_piece(const uint4 &q, Sum &sum) {
    float2 s = both(0.f);
    float amax = 0.f;
    pairs<TYPE>(q, [&](float2 v) {
        s = fma2(v, v, s);
        amax = fmaxf(amax, fmaxf(fabsf(v.x), fabsf(v.y)));
    });
    if (amax > 0x1p40f || (amax < 0x1p-56f && amax != 0.f)) {              // as in add_squares
        const float2 shift = both(amax > 1.f ? 0x1p-70f : 0x1p90f);
        s = both(0.f);
        pairs<TYPE>(q, [&](float2 v) {
            v = mul2(v, shift);
            s = fma2(v, v, s);
        });
        sum.rest += (double)(s.x + s.y) * (amax > 1.f ? 0x1p140 : 0x1p-180);
    } else {
        sum.add(s.x + s.y);
    }
}
// A piece scaled, element k of it the tensor's element `at` + k
template <int TYPE>
__device__ __forceinline__ void scale_piece(const Entry &e, const uint4 &q, int64_t at, const Factor &factor) {
    float v[8];
    int n = 0;
    pairs<TYPE>(q, [&](float2 f) {
        v[n++] = factor(f.x);
        v[n++] = factor(f.y);
    });
    constexpr int SIZE = TYPE == GEMM_F32 ? 4 : 2;
    if (e.apart) {
#pragma unroll
        for (int k = 0; k < 16 / SIZE; ++k) store_one(e.c, TYPE, at + k, v[k]);
        return;
    }
    uint4 *to = reinterpret_cast<uint4 *>(e.c + at * SIZE);
    if constexpr (TYPE == GEMM_F32)
        *to = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    else if constexpr (TYPE == GEMM_BF16) *to = pack8(static_cast<const __nv_bfloat16 *>(nullptr), v);
    else *to = pack8(static_cast<const __half *>(nullptr), v);
}

template <int N>
__global__ void __launch_bounds__(THREADS)
    clip_few_kernel(const __grid_constant__ Table<N, FEW_CTAS> t, float limit, float *norm_out) {
    __shared__ Part sums[FEW_CTAS];
    const Range r = range_of(t.rows, blockIdx.x, FEW_CTAS);
    const int thread = threadIdx.x, warp = thread / 32, lane = thread % 32;
    uint4 q[FEW_HELD];
    int owner[FEW_HELD];                                   // the row's tensor, -1 past the range
    int64_t at[FEW_HELD];                                  // the piece's first element, -1 where there is none
    int64_t edge = -1;                                     // the thread's element outside the pieces
    int edge_owner = 0;
    float edge_value = 0.f;
    int i = t.start[blockIdx.x];
    cluster_arrive();                                      // (waited for before the stores: none goes to a CTA that has not begun)
    wait_for_previous();
    let_next_launch();
#pragma unroll
    for (int k = 0; k < FEW_HELD; ++k) {
        const uint32_t row = r.begin + k;
        owner[k] = -1;
        at[k] = -1;
        q[k] = make_uint4(0, 0, 0, 0);
        if (row >= r.end) continue;
        while (i + 1 < t.count && t.e[i + 1].first <= row) ++i;
        const Entry &e = t.e[i];
        const Span s(e);
        const int64_t piece = (int64_t)(row - e.first) * THREADS + thread;
        owner[k] = i;
        if (piece < s.pieces) {
            at[k] = s.head + piece * (e.type == GEMM_F32 ? 4 : 8);
            q[k] = *reinterpret_cast<const uint4 *>(e.g + at[k] * (e.type == GEMM_F32 ? 4 : 2));
        }
        if (k == warp && row == e.first) {                 // lanes 0 to 6: before the pieces, 16 to 22: behind them
            if (lane < s.head) edge = lane;
            if (lane >= 16 && lane - 16 < s.tail) edge = e.n - s.tail + (lane - 16);
            edge_owner = i;
        }
    }
    if (edge >= 0) edge_value = load_one(t.e[edge_owner].g, t.e[edge_owner].type, edge);
    Sum sum;
#pragma unroll
    for (int k = 0; k < FEW_HELD; ++k) {
        if (owner[k] < 0) break;
        const int type = t.e[owner[k]].type;
        if (type == GEMM_F32) add_piece<GEMM_F32>(q[k], sum);
        else if (type == GEMM_BF16) add_piece<GEMM_BF16>(q[k], sum);
        else add_piece<GEMM_F16>(q[k], sum);
    }
    add_square(edge_value, sum);
    sum = block_sum(sum);
    cluster_wait();
    if (thread < FEW_CTAS) {
        uint32_t to;
        asm("mapa.shared::cluster.u32 %0, %1, %2;"
            : "=r"(to)
            : "r"((uint32_t)__cvta_generic_to_shared(&sums[blockIdx.x])), "r"(thread));
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(sum.high), "f"(sum.low) : "memory");
        asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(to + 8), "d"(sum.rest) : "memory");
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    Sum all;
#pragma unroll
    for (int k = 0; k < FEW_CTAS; ++k) all.add(sums[k]);
    float norm;
    const Factor factor = factor_of(all, limit, norm);
    if (blockIdx.x == 0 && thread == 0) *norm_out = norm;
    auto written = [&](const Entry &e) { return e.c && !(factor.one && e.c == e.g); };
#pragma unroll
    for (int k = 0; k < FEW_HELD; ++k) {
        if (at[k] < 0) continue;
        const Entry &e = t.e[owner[k]];
        if (!written(e)) continue;
        if (e.type == GEMM_F32) scale_piece<GEMM_F32>(e, q[k], at[k], factor);
        else if (e.type == GEMM_BF16) scale_piece<GEMM_BF16>(e, q[k], at[k], factor);
        else scale_piece<GEMM_F16>(e, q[k], at[k], factor);
    }
    if (edge >= 0) {
        const Entry &e = t.e[edge_owner];
        if (written(e)) store_one(e.c, e.type, edge, factor(edge_value));
    }
}

// ------------------------------------------------------------------------------------------- launches

// Tables by size: a launch copies all of its own
constexpr int SMALL = 32, MIDDLE = 256, LARGE = 900;

int64_t rows_of(const gemm_clip_tensor &t) {               // at least one for a tensor that is not empty
    const int64_t bytes = t.n * (t.type == GEMM_F32 ? 4 : 2);
    return t.n == 0 ? 0 : std::max<int64_t>(1, (bytes + ROW - 1) / ROW);
}

struct Call {
    const gemm_clip_tensor *tensors;
    int64_t count;
    float limit;
    float *norm;
    Part *parts;
    int sms;
    cudaStream_t stream;
};

// Up to FEW_ROWS rows go to the single cluster: one launch where the host's two would be what a call costs
template <int N, int M>
cudaError_t clip_few(const Call &k, const Table<M> &from) {
    Table<N, FEW_CTAS> t;
    t.count = from.count;
    t.rows = from.rows;
    t.copies = from.copies;
    std::copy(from.start, from.start + FEW_CTAS, t.start);
    std::copy(from.e, from.e + from.count, t.e);
    const Launch c(FEW_CTAS, THREADS, 0, FEW_CTAS, k.stream);
    return cudaLaunchKernelEx(&c.config, clip_few_kernel<N>, t, k.limit, k.norm);
}

// A list too large for L2: of what the first kernel reads the last KEEP_BYTES stay there, and what the second one is through
// with leaves first.  100.7 million fp32 values 190 us, 195 without (48 million bytes 192); 291 tensors 62 and 66.
// The stores' part of it alone costs 1 %.
constexpr int64_t L2_BYTES = 60000000, KEEP_BYTES = 96000000;

// CTAs of a list with little for each: with two per SM the second kernel's are on the SMs, and wait, before the first kernel's
// leave, with five (of 48 registers a thread) they are not, 5 us in all.  One tensor of a million bf16 values 7.3 us, 11.5 with
// five, 8 million 13.0 and 16.2; 300 tensors of 1 million 12.1 and 14.1, of 4 million 18.4 and 17.2.  A tensor counts as two steps
// beside its own: its first and last elements.
constexpr int FEW_PER_SM = 2, FEW_STEPS = 8;
uint32_t ctas_of(uint32_t rows, int64_t steps, int count, int sms) {
    const int most = std::min((steps + 2 * count <= FEW_STEPS * sms ? FEW_PER_SM : CTAS_PER_SM) * sms, MAX_PARTS);
    return std::min(std::max(1u, rows), (uint32_t)most);
}

// The tensors in launches of up to N: all norms' kernels, then all scalings'
template <int N>
cudaError_t clip(const Call &k) {
    const int64_t launches = std::max<int64_t>(1, (k.count + N - 1) / N);
    Table<N> t;
    int parts = 0, grid = 0;
    bool any = false, few = false, large = false;
    auto table = [&](int64_t l) {
        t.count = 0;
        t.rows = 0;
        t.copies = false;
        int64_t steps = 0;
        const int64_t first = l * N, last = std::min<int64_t>(first + N, k.count);
        for (int64_t i = first; i < last; ++i) {
            const gemm_clip_tensor &from = k.tensors[i];
            if (from.n == 0) continue;
            const uintptr_t apart = reinterpret_cast<uintptr_t>(from.g) ^ reinterpret_cast<uintptr_t>(from.c);
            t.e[t.count++] = Entry{static_cast<const uint8_t *>(from.g), static_cast<uint8_t *>(from.c), from.n, t.rows,
                                   (int16_t)from.type, (int16_t)((apart & 15) != 0)};
            const int64_t rows = rows_of(from);
            t.rows += (uint32_t)rows;
            steps += (rows + STEP - 1) / STEP;
            t.copies = t.copies || (from.c && from.c != from.g);
            any = any || from.c;
        }
        few = launches == 1 && t.rows <= FEW_ROWS;
        large = launches == 1 && (int64_t)t.rows * ROW > L2_BYTES;
        grid = few ? FEW_CTAS : (int)ctas_of(t.rows, steps, t.count, k.sms);
        for (int b = 0, i = 0; b < grid; ++b) {
            const uint32_t begin = range_of(t.rows, (uint32_t)b, (uint32_t)grid).begin;
            while (i + 1 < t.count && t.e[i + 1].first <= begin) ++i;
            t.start[b] = (uint16_t)i;
        }
    };
    for (int64_t l = 0; l < launches; ++l) {
        table(l);
        if (few) return t.count <= 16 ? clip_few<16>(k, t) : clip_few<FEW_ROWS>(k, t);      // (a tensor has a row at least)
        const cudaError_t e = launch(clip_norm_kernel<N>, grid, THREADS, 0, k.stream, t, k.parts, parts,
                                     large ? (uint32_t)(KEEP_BYTES / ROW / grid) : ~0u);
        if (e != cudaSuccess) return e;
        parts = std::max(parts, grid);
    }
    for (int64_t l = 0; l < launches; ++l) {
        if (launches > 1) table(l);
        if (!any) {                                        // the norm alone
            t.count = 0;
            t.rows = 0;
            grid = 1;
        }
        const cudaError_t e = launch(clip_scale_kernel<N>, grid, THREADS, 0, k.stream, t, (const Part *)k.parts, parts, k.limit,
                                     l == 0 ? k.norm : (float *)nullptr, large);
        if (e != cudaSuccess || !any) return e;
    }
    return cudaSuccess;
}

}  // namespace
}  // namespace gb300

using namespace gb300;

extern "C" gemm_status gemm_clip_run(int64_t count, const gemm_clip_tensor *tensors, float limit, float *NORM, void *workspace,
                                     size_t workspace_bytes, void *cuda_stream) {
    if (count < 0 || !(limit >= 0.f) || (count > 0 && !tensors) || !NORM || !workspace || workspace_bytes < GEMM_CLIP_WORKSPACE)
        return GEMM_ERR_INVALID_ARG;
    int64_t rows = 0;
    for (int64_t i = 0; i < count; ++i) {
        const gemm_clip_tensor &t = tensors[i];
        if (t.n < 0 || t.n > (int64_t)1 << 40 || (t.n > 0 && !t.g)) return GEMM_ERR_INVALID_ARG;
        if (t.type != GEMM_F32 && t.type != GEMM_BF16 && t.type != GEMM_F16) return GEMM_ERR_UNSUPPORTED;
        const uintptr_t size = t.type == GEMM_F32 ? 4 : 2;
        if (reinterpret_cast<uintptr_t>(t.g) % size || reinterpret_cast<uintptr_t>(t.c) % size) return GEMM_ERR_ALIGNMENT;
        rows += rows_of(t);
        if (rows > INT32_MAX) return GEMM_ERR_UNSUPPORTED;
    }
    if (reinterpret_cast<uintptr_t>(NORM) % 4 || !rows::aligned16(workspace)) return GEMM_ERR_ALIGNMENT;
    int sms = 0;
    const gemm_status st = rows::device_sms(&sms);
    if (st != GEMM_OK) return st;
    const Call k{tensors, count, limit, NORM, static_cast<Part *>(workspace), sms, reinterpret_cast<cudaStream_t>(cuda_stream)};
    const cudaError_t e = count <= SMALL ? clip<SMALL>(k) : count <= MIDDLE ? clip<MIDDLE>(k) : clip<LARGE>(k);
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}
