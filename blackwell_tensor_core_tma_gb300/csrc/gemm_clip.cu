// The Euclidean norm of many tensors together, and the tensors scaled to a largest norm (gemm_clip_run in
// include/gb300gemm.h):
//
//   norm = sqrt(sum g^2),  c = g * min(1, limit / norm)
//
// Two kernels over the same chunks of CHUNK bytes.  The first leaves each CTA's sum of squares; in the second every CTA adds
// those up, in the same order, so that no counter or second launch stands between them, and scales its chunks, the last
// ones first: what the first kernel read last is still in L2.
//
// A thread's sixteen-byte pieces of a chunk are squared and summed in fp32, scaled by a power of two where their
// largest magnitude is far from one (a square stays within fp32's range), and everything above that is summed in 64 bits:
// one 64-bit operation for 32 or 64 values, which the unit's rate has room for.
#include <algorithm>

#include "gemm_rows.cuh"

namespace gb300 {
namespace {

using namespace rows;

constexpr int THREADS = 256;
constexpr int PER_THREAD = 8;                              // 16-byte pieces of a chunk
constexpr int CHUNK = THREADS * PER_THREAD * 16;           // bytes
constexpr int MAX_PARTS = GEMM_CLIP_WORKSPACE / (int)sizeof(double);

struct Entry {
    const uint8_t *g;
    uint8_t *c;
    int64_t n;
    uint32_t first;          // its first chunk
    int16_t type;
    int16_t apart;           // c is not a multiple of 16 bytes from g: written element by element
};
// The tensors of one launch, by value: a captured graph keeps them
template <int N>
struct Table {
    int count;
    uint32_t chunks;
    Entry e[N];
};

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
    int64_t head, pieces, tail;
    __device__ __forceinline__ Span(const Entry &e) {
        const int size = e.type == GEMM_F32 ? 4 : 2, per = 16 / size;
        head = (int64_t)((16 - (reinterpret_cast<uintptr_t>(e.g) & 15)) & 15) / size;
        if (head > e.n) head = e.n;
        pieces = (e.n - head) / per;
        tail = e.n - head - pieces * per;
    }
};

template <int N>
__device__ __forceinline__ int entry_of(const Table<N> &t, uint32_t chunk) {      // the last one that begins at or before it
    int low = 0, high = t.count - 1;
    while (low < high) {
        const int mid = (low + high + 1) / 2;
        if (t.e[mid].first <= chunk) low = mid; else high = mid - 1;
    }
    return low;
}

// f(pair of values) for a piece
template <typename F>
__device__ __forceinline__ void each(const uint4 &q, int type, F f) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (type == GEMM_F32) {
            f(__uint_as_float(w[i]));
        } else if (type == GEMM_BF16) {
            f(__uint_as_float(w[i] << 16));
            f(__uint_as_float(w[i] & 0xFFFF0000u));
        } else {
            const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            f(v.x);
            f(v.y);
        }
    }
}

// The power of two that brings values of this largest magnitude to where their squares, and 64 of them together, are within
// fp32's range with room below: fp32 loses nothing that counts beside the largest square
__device__ __forceinline__ float shift_of(float amax) { return amax > 0x1p60f ? 0x1p-70f : amax < 0x1p-40f ? 0x1p100f : 1.f; }
__device__ __forceinline__ double unshifted(float sum, float shift) {
    const double back = shift == 1.f ? 1.0 : shift < 1.f ? 0x1p140 : 0x1p-200;
    return (double)sum * back;
}
__device__ __forceinline__ double square_of(float v) { return (double)v * (double)v; }

__device__ __forceinline__ double block_sum(double v) {            // the same order every time; valid in all threads
    __shared__ double s[THREADS / 32];
#pragma unroll
    for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x / 32] = v;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) t += s[i];
    return t;
}

template <int TYPE>
__device__ __forceinline__ double squares(const uint4 *g, int64_t pieces) {
    uint4 q[PER_THREAD];
#pragma unroll
    for (int i = 0; i < PER_THREAD; ++i) {
        const int64_t at = i * THREADS + threadIdx.x;
        q[i] = at < pieces ? g[at] : make_uint4(0, 0, 0, 0);
    }
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < PER_THREAD; ++i) each(q[i], TYPE, [&](float v) { amax = fmaxf(amax, fabsf(v)); });
    const float shift = shift_of(amax);
    float sum[4] = {};
#pragma unroll
    for (int i = 0; i < PER_THREAD; ++i) {
        float &s = sum[i % 4];
        each(q[i], TYPE, [&](float v) { v *= shift; s = fmaf(v, v, s); });
    }
    return unshifted((sum[0] + sum[1]) + (sum[2] + sum[3]), shift);
}

template <int N>
__global__ void __launch_bounds__(THREADS) clip_norm_kernel(const __grid_constant__ Table<N> t, double *parts) {
    wait_for_previous();
    let_next_launch();
    double sum = 0.0;
    for (uint32_t chunk = blockIdx.x; chunk < t.chunks; chunk += gridDim.x) {
        const Entry &e = t.e[entry_of(t, chunk)];
        const Span s(e);
        const int size = e.type == GEMM_F32 ? 4 : 2;
        const uint32_t c = chunk - e.first;
        const int64_t at = (int64_t)c * (THREADS * PER_THREAD);
        const uint4 *g = reinterpret_cast<const uint4 *>(e.g + s.head * size) + at;
        if (e.type == GEMM_F32) sum += squares<GEMM_F32>(g, s.pieces - at);
        else if (e.type == GEMM_BF16) sum += squares<GEMM_BF16>(g, s.pieces - at);
        else sum += squares<GEMM_F16>(g, s.pieces - at);
        if (c == 0) {                                      // at most seven elements before and behind the pieces
            if (threadIdx.x < s.head) sum += square_of(load_one(e.g, e.type, threadIdx.x));
            if (threadIdx.x < s.tail) sum += square_of(load_one(e.g, e.type, e.n - s.tail + threadIdx.x));
        }
    }
    sum = block_sum(sum);
    if (threadIdx.x == 0) parts[blockIdx.x] = sum;
}

// limit / norm as a product of two: where it is below fp32's normal numbers' upper part, a power of two and the rest
struct Factor {
    float rest, power;
    __device__ __forceinline__ float operator()(float v) const { return v * power * rest; }
};

template <int TYPE>
__device__ __forceinline__ void scale(const uint4 *g, uint4 *c, int64_t pieces, const Factor &factor) {
    uint4 q[PER_THREAD];
#pragma unroll
    for (int i = 0; i < PER_THREAD; ++i) {
        const int64_t at = i * THREADS + threadIdx.x;
        q[i] = at < pieces ? g[at] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < PER_THREAD; ++i) {
        const int64_t at = i * THREADS + threadIdx.x;
        float v[8];
        int n = 0;
        each(q[i], TYPE, [&](float f) { v[n++] = factor(f); });
        if (at < pieces) {
            if constexpr (TYPE == GEMM_F32)
                c[at] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
            else if constexpr (TYPE == GEMM_BF16) c[at] = pack8(static_cast<const __nv_bfloat16 *>(nullptr), v);
            else c[at] = pack8(static_cast<const __half *>(nullptr), v);
        }
    }
}

template <int N>
__global__ void __launch_bounds__(THREADS)
    clip_scale_kernel(const __grid_constant__ Table<N> t, const double *parts, int n, float limit, float *norm_out) {
    wait_for_previous();
    let_next_launch();
    double sum = 0.0;
    for (int i = threadIdx.x; i < n; i += THREADS) sum += parts[i];
    const double norm = sqrt(block_sum(sum));
    if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
    // a norm that is not a number makes a factor that is none
    const double ratio = norm <= (double)limit ? 1.0 : (double)limit / norm;
    const float power = ratio < 0x1p-100 ? 0x1p-100f : 1.f;
    const Factor factor{(float)(ratio / (double)power), power};
    for (uint32_t i = blockIdx.x; i < t.chunks; i += gridDim.x) {
        const uint32_t chunk = t.chunks - 1 - i;
        const Entry &e = t.e[entry_of(t, chunk)];
        if (!e.c || (ratio == 1.0 && e.c == e.g)) continue;
        const Span s(e);
        const int size = e.type == GEMM_F32 ? 4 : 2;
        const uint32_t c = chunk - e.first;
        const int64_t at = (int64_t)c * (THREADS * PER_THREAD);
        if (e.apart) {
            const int64_t per = 16 / size, first = s.head + at * per;
            const int64_t last = min(s.head + s.pieces * per, first + THREADS * PER_THREAD * per);
            for (int64_t k = first + threadIdx.x; k < last; k += THREADS)
                store_one(e.c, e.type, k, factor(load_one(e.g, e.type, k)));
        } else {
            const uint4 *g = reinterpret_cast<const uint4 *>(e.g + s.head * size) + at;
            uint4 *to = reinterpret_cast<uint4 *>(e.c + s.head * size) + at;
            if (e.type == GEMM_F32) scale<GEMM_F32>(g, to, s.pieces - at, factor);
            else if (e.type == GEMM_BF16) scale<GEMM_BF16>(g, to, s.pieces - at, factor);
            else scale<GEMM_F16>(g, to, s.pieces - at, factor);
        }
        if (c == 0) {
            if (threadIdx.x < s.head) store_one(e.c, e.type, threadIdx.x, factor(load_one(e.g, e.type, threadIdx.x)));
            if (threadIdx.x < s.tail) {
                const int64_t k = e.n - s.tail + threadIdx.x;
                store_one(e.c, e.type, k, factor(load_one(e.g, e.type, k)));
            }
        }
    }
}

// Tables by size: a launch copies all of its own
constexpr int SMALL = 32, MIDDLE = 256, LARGE = 1000;

int64_t chunks_of(const gemm_clip_tensor &t) {             // at least one for a tensor that is not empty
    const int64_t bytes = t.n * (t.type == GEMM_F32 ? 4 : 2);
    return t.n == 0 ? 0 : std::max<int64_t>(1, (bytes + CHUNK - 1) / CHUNK);
}

template <int N>
void fill(Table<N> &t, const gemm_clip_tensor *tensors, int64_t count) {
    t.count = 0;
    t.chunks = 0;
    for (int64_t i = 0; i < count; ++i) {
        const gemm_clip_tensor &from = tensors[i];
        if (from.n == 0) continue;
        const uintptr_t apart = reinterpret_cast<uintptr_t>(from.g) ^ reinterpret_cast<uintptr_t>(from.c);
        t.e[t.count++] = Entry{static_cast<const uint8_t *>(from.g), static_cast<uint8_t *>(from.c), from.n, t.chunks,
                               (int16_t)from.type, (int16_t)((apart & 15) != 0)};
        t.chunks += (uint32_t)chunks_of(from);
    }
}

struct Call {
    const gemm_clip_tensor *tensors;
    int64_t count;
    float limit;
    float *norm;
    double *parts;
    int sms;
    cudaStream_t stream;
};

// The tensors in launches of up to N: all norms' kernels, then all scalings'
template <int N>
cudaError_t clip(const Call &k) {
    const int launches = (int)std::max<int64_t>(1, (k.count + N - 1) / N);
    const int most = std::max(1, std::min(4 * k.sms, MAX_PARTS / launches));
    Table<N> t;
    int parts = 0;
    bool any = false;
    auto table = [&](int l) {
        const int64_t first = (int64_t)l * N;
        fill(t, k.tensors + first, std::min<int64_t>(N, k.count - first));
    };
    for (int l = 0; l < launches; ++l) {
        table(l);
        for (int i = 0; i < t.count; ++i) any = any || t.e[i].c;
        const int grid = (int)std::min<uint32_t>(std::max(1u, t.chunks), (uint32_t)most);
        const cudaError_t e = launch(clip_norm_kernel<N>, grid, THREADS, 0, k.stream, t, k.parts + parts);
        if (e != cudaSuccess) return e;
        parts += grid;
    }
    for (int l = 0; l < launches; ++l) {
        if (launches > 1) table(l);
        if (!any) t.chunks = 0;                            // the norm alone
        const int grid = (int)std::min<uint32_t>(std::max(1u, t.chunks), (uint32_t)(4 * k.sms));
        const cudaError_t e = launch(clip_scale_kernel<N>, grid, THREADS, 0, k.stream, t, (const double *)k.parts, parts, k.limit,
                                     l == 0 ? k.norm : (float *)nullptr);
        if (e != cudaSuccess) return e;
        if (!any) break;
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
    if (count > (int64_t)LARGE * MAX_PARTS) return GEMM_ERR_UNSUPPORTED;
    int64_t chunks = 0;
    for (int64_t i = 0; i < count; ++i) {
        const gemm_clip_tensor &t = tensors[i];
        if (t.n < 0 || t.n > (int64_t)1 << 40 || (t.n > 0 && !t.g)) return GEMM_ERR_INVALID_ARG;
        if (t.type != GEMM_F32 && t.type != GEMM_BF16 && t.type != GEMM_F16) return GEMM_ERR_UNSUPPORTED;
        const uintptr_t size = t.type == GEMM_F32 ? 4 : 2;
        if (reinterpret_cast<uintptr_t>(t.g) % size || reinterpret_cast<uintptr_t>(t.c) % size) return GEMM_ERR_ALIGNMENT;
        chunks += chunks_of(t);
    }
    if (chunks > INT32_MAX) return GEMM_ERR_UNSUPPORTED;
    if (reinterpret_cast<uintptr_t>(NORM) % 4 || !rows::aligned16(workspace)) return GEMM_ERR_ALIGNMENT;
    int sms = 0;
    const gemm_status st = rows::device_sms(&sms);
    if (st != GEMM_OK) return st;
    const Call k{tensors, count, limit, NORM, static_cast<double *>(workspace), sms, reinterpret_cast<cudaStream_t>(cuda_stream)};
    const cudaError_t e = count <= SMALL ? clip<SMALL>(k) : count <= MIDDLE ? clip<MIDDLE>(k) : clip<LARGE>(k);
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}
