// Root-mean-square norm with the residual's addition, and its gradient (gemm_norm_run,
// gemm_norm_backward in include/gb300gemm.h).
//
//   h = round(x + r),  rstd = 1 / sqrt(mean_k h^2 + eps),  y = h * rstd * w
//   n = h * rstd,  g = dy * w,  dx = dh + rstd * (g - n * mean_k(g * n)),  dw = sum_rows dy * n
//
// One pass over memory: a row lives in the registers of its threads (U units of eight elements each)
// between the sum that the statistics need and the outputs that use them.
#include <initializer_list>
#include <mutex>
#include <type_traits>

#include "gemm_rows.cuh"

namespace gb300 {
namespace rows {

gemm_status device_sms(int *sms) {
    constexpr int MAX_DEVICES = 64;
    static int known[MAX_DEVICES];          // 0: not asked yet, -1: not a GB300
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= MAX_DEVICES) return GEMM_ERR_CUDA;
    std::lock_guard<std::mutex> lock(mu);
    if (known[dev] == 0) {
        int major = 0, minor = 0, n = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
            return GEMM_ERR_CUDA;
        known[dev] = major == 10 && minor == 3 ? n : -1;
    }
    if (known[dev] < 0) return GEMM_ERR_UNSUPPORTED;
    *sms = known[dev];
    return GEMM_OK;
}

}  // namespace rows

namespace {

using namespace rows;

constexpr int MAX_K = 32768;         // a row in registers: 1024 threads x 4 units
constexpr int UNIT = 8;              // elements: 16-byte accesses of 16-bit types, a warp's contiguous
constexpr int MAX_WARPS = 32;

// How a row is spread over threads: U units per thread, `tpr` threads per row (a power of two up to
// 32, else whole warps), `rpc` rows per CTA.
struct RowShape {
    int u, tpr, rpc;
};
RowShape row_shape(int units, int u) {
    RowShape s;
    s.u = u;
    const int need = (units + s.u - 1) / s.u;
    if (need <= 32) {
        s.tpr = 4;
        while (s.tpr < need) s.tpr *= 2;
    } else {
        s.tpr = (need + 31) / 32 * 32;
    }
    s.rpc = s.tpr >= 256 ? 1 : 256 / s.tpr;
    return s;
}

// Sum over the threads of a row (threadIdx.y), the same in each of them and in a fixed order: within a warp,
// then each warp over the row's warps.  Every thread of the CTA takes part.  `red` holds one float per warp; it may
// be written again after the next __syncthreads.
__device__ __forceinline__ float row_sum(float v, float *red) {
    const int tpr = blockDim.x;
    for (int o = min(tpr, 32) / 2; o > 0; o /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (tpr <= 32) return v;
    const int lane = threadIdx.x & 31, warps = tpr / 32;
    if (lane == 0) red[threadIdx.y * warps + threadIdx.x / 32] = v;
    __syncthreads();
    v = lane < warps ? red[threadIdx.y * warps + lane] : 0.f;
    for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

struct NormParams {
    const void *x, *r;
    const float *w;
    void *h, *y;
    uint8_t *sf;
    float *rstd;
    int64_t M;
    int K;
    float eps;
};

// One row per group of threads (threadIdx.y): all of its loads are requested before the first is used.
template <typename XT, typename HT, typename YT, int U>
__global__ void __launch_bounds__(U == 4 ? 1024 : 512) norm_kernel(const __grid_constant__ NormParams p) {
    constexpr int N = UNIT, PX = PIECES<XT, N>, PH = PIECES<HT, N>;
    __shared__ float red[MAX_WARPS];
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int units = p.K / N, tpr = blockDim.x;
    const XT *x = static_cast<const XT *>(p.x) + row * p.K;
    const HT *r = static_cast<const HT *>(p.r) + row * p.K;
    HT *h = static_cast<HT *>(p.h) + row * p.K;

    uint4 xq[U][PX], rq[U][PH];
    bool on[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
        const int u = threadIdx.x + j * tpr;
        on[j] = row < p.M && u < units;
        load_pieces(x + u * N, on[j], xq[j]);
        load_pieces(r + u * N, on[j] && p.r, rq[j]);
    }
    float v[U][N];
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < U; ++j) {
        float a[N];
        unpack(x, xq[j], v[j]);
        unpack(r, rq[j], a);
#pragma unroll
        for (int i = 0; i < N; ++i) v[j][i] += a[i];
        // the norm takes the rounded h, so that the gradient from a stored h is the gradient of
        // what was computed
        round_store(h + (threadIdx.x + j * tpr) * N, on[j] && p.h, v[j]);
#pragma unroll
        for (int i = 0; i < N; ++i) sum = fmaf(v[j][i], v[j][i], sum);
    }
    sum = row_sum(sum, red);
    const float rstd = __frsqrt_rn(sum / (float)p.K + p.eps);
    if (row < p.M && threadIdx.x == 0 && p.rstd) p.rstd[row] = rstd;

#pragma unroll
    for (int j = 0; j < U; ++j) {
        const int u = threadIdx.x + j * tpr;
        if (on[j]) {
            float w[N];
            load(p.w + u * N, w);
#pragma unroll
            for (int i = 0; i < N; ++i) v[j][i] = v[j][i] * rstd * w[i];
        }
        if constexpr (sizeof(YT) == 1) {
            const uint32_t code = quantise(v[j], static_cast<uint8_t *>(p.y) + row * p.K + u * N, on[j]);
            if (on[j] && u % (BLOCK / N) == 0) p.sf[row * ((p.K + BLOCK - 1) / BLOCK) + u / (BLOCK / N)] = (uint8_t)code;
        } else if (on[j]) {
            store(static_cast<YT *>(p.y) + row * p.K + u * N, v[j]);
        }
    }
}

// Rows ahead come through a ring in shared memory by asynchronous copies.  Every thread copies the very units that it
// reads, so the ring needs no barrier of its own.
constexpr int MAX_STAGES = 4;
// `part`: the lanes' pieces are 32 bytes apart, so half of each sector is another copy's: keep it in L1 for that
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool part) {
    if (part) asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 load_shared4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void wait_stage(int stages) {         // all but the last stages - 1 groups have landed
    if (stages == 4) asm volatile("cp.async.wait_group 3;" ::: "memory");
    else if (stages == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (stages == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
}


struct NormBackParams {
    const void *dy, *dh, *h;
    const float *rstd, *w;
    void *dx, *y;
    float *parts;        // one row of K per CTA, or null when dw is not wanted
    int64_t M;
    int K;
    float inverse_k;
    int stages;          // rows of the ring (up to MAX_STAGES), or 0: a row does not fit, and is loaded where it is used
};

// A CTA walks rows (rpc at a time) with dw in registers; a row costs one barrier, that of its sum.
template <typename GT, typename HT, typename YT, int U, int THREADS>
__global__ void __launch_bounds__(THREADS, U == 1 ? 2 : 1) norm_back_kernel(const __grid_constant__ NormBackParams p) {
    extern __shared__ uint4 ring[];                    // [stages][pieces of a unit: dy, h, dh][U][threads]
    __shared__ float red[2][MAX_WARPS];
    constexpr int PG = PIECES<GT, UNIT>, PH = PIECES<HT, UNIT>, PER_UNIT = PG + 2 * PH;
    constexpr bool KEEP = THREADS == 512;                      // g and n stay in registers over the sum; else they are read again
    constexpr bool KEEP_W = U <= 2;
    const int units = p.K / UNIT, tpr = blockDim.x, threads = tpr * blockDim.y, tid = threadIdx.y * tpr + threadIdx.x;
    const uint32_t mine = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + tid * 16;
    const uint32_t unit_bytes = threads * 16, stage_bytes = PER_UNIT * U * unit_bytes;

    const GT *dy = static_cast<const GT *>(p.dy);
    const HT *h = static_cast<const HT *>(p.h), *dh = static_cast<const HT *>(p.dh);
    auto request = [&](int64_t row, int slot) {
        if (row < p.M) {
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int u = threadIdx.x + j * tpr;
                if (u >= units) continue;
                const int64_t at = row * p.K + u * UNIT;
                const uint32_t to = mine + slot * stage_bytes + j * unit_bytes;
#pragma unroll
                for (int i = 0; i < PG; ++i) copy16(to + i * U * unit_bytes, dy + at + i * 4, PG > 1);
#pragma unroll
                for (int i = 0; i < PH; ++i) copy16(to + (PG + i) * U * unit_bytes, h + at + i * 4, PH > 1);
                if (dh) {
#pragma unroll
                    for (int i = 0; i < PH; ++i) copy16(to + (PG + PH + i) * U * unit_bytes, dh + at + i * 4, PH > 1);
                }
            }
        }
        copies_commit();
    };
    auto read = [&](auto *from, int64_t row, int slot, int j, int piece, float (&v)[UNIT]) {      // piece: of the ring
        using T = std::remove_const_t<std::remove_pointer_t<decltype(from)>>;
        if (p.stages == 0) {
            load(from + row * p.K + (threadIdx.x + j * tpr) * UNIT, v);
            return;
        }
        uint4 q[PIECES<T, UNIT>];
#pragma unroll
        for (int i = 0; i < PIECES<T, UNIT>; ++i) q[i] = load_shared4(mine + slot * stage_bytes + ((piece + i) * U + j) * unit_bytes);
        unpack(from, q, v);
    };
    float dw[U][UNIT];
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
        for (int i = 0; i < UNIT; ++i) dw[j][i] = 0.f;

    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    const int64_t own = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;      // this thread's first row
    for (int s = 0; s < p.stages; ++s) request(own + s * step, s);
    float w[KEEP_W ? U : 1][UNIT];
    if (KEEP_W) {
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (threadIdx.x + j * tpr < units) load(p.w + (threadIdx.x + j * tpr) * UNIT, w[j]);
    }
    float next_rstd = own < p.M ? p.rstd[own] : 0.f;     // a row ahead, so that no row waits for it
    int turn = 0, slot = 0;
    for (int64_t row = own; row - threadIdx.y < p.M; row += step, turn ^= 1) {
        const bool live = row < p.M;
        const float rstd = next_rstd;
        next_rstd = row + step < p.M ? p.rstd[row + step] : 0.f;
        if (p.stages) wait_stage(p.stages);
        float g[KEEP ? U : 1][UNIT], n[KEEP ? U : 1][UNIT];
        float sum = 0.f, sum2 = 0.f;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int u = threadIdx.x + j * tpr, k = KEEP ? j : 0, kw = KEEP_W ? j : 0;
            if (live && u < units) {
                read(dy, row, slot, j, 0, g[k]);
                read(h, row, slot, j, PG, n[k]);
                if (!KEEP_W) load(p.w + u * UNIT, w[kw]);
#pragma unroll
                for (int i = 0; i < UNIT; ++i) {
                    n[k][i] *= rstd;
                    dw[j][i] = fmaf(g[k][i], n[k][i], dw[j][i]);
                    g[k][i] *= w[kw][i];
                    (i & 1 ? sum2 : sum) = fmaf(g[k][i], n[k][i], i & 1 ? sum2 : sum);
                }
                if (p.y) {
                    float y[UNIT];
#pragma unroll
                    for (int i = 0; i < UNIT; ++i) y[i] = n[k][i] * w[kw][i];
                    store(static_cast<YT *>(p.y) + row * p.K + u * UNIT, y);
                }
            }
        }
        const float c = row_sum(sum + sum2, red[turn]) * p.inverse_k;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int u = threadIdx.x + j * tpr, k = KEEP ? j : 0, kw = KEEP_W ? j : 0;
            if (live && u < units) {
                if (!KEEP) {
                    read(dy, row, slot, j, 0, g[k]);
                    read(h, row, slot, j, PG, n[k]);
                    if (!KEEP_W) load(p.w + u * UNIT, w[kw]);
#pragma unroll
                    for (int i = 0; i < UNIT; ++i) {
                        n[k][i] *= rstd;
                        g[k][i] *= w[kw][i];
                    }
                }
                float d[UNIT];
                if (dh) {
                    read(dh, row, slot, j, PG + PH, d);
                } else {
#pragma unroll
                    for (int i = 0; i < UNIT; ++i) d[i] = 0.f;
                }
#pragma unroll
                for (int i = 0; i < UNIT; ++i) d[i] += rstd * (g[k][i] - n[k][i] * c);
                store(static_cast<HT *>(p.dx) + row * p.K + u * UNIT, d);
            }
        }
        if (p.stages) request(row + p.stages * step, slot);          // the thread itself has read what lay there
        slot = slot + 1 >= p.stages ? 0 : slot + 1;
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (!p.parts) return;

    // the CTA's sums in a fixed order: rows of threads first, then (norm_dw_kernel) CTAs
    float *part = p.parts + (int64_t)blockIdx.x * p.K;
    if (blockDim.y == 1) {
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int u = threadIdx.x + j * tpr;
            if (u < units) store(part + u * UNIT, dw[j]);
        }
        return;
    }
    float *shared = reinterpret_cast<float *>(ring);     // no copy is under way: the last requests were empty
    __syncthreads();
#pragma unroll
    for (int j = 0; j < U; ++j) {
        const int u = threadIdx.x + j * tpr;
        if (u < units) store(shared + threadIdx.y * p.K + u * UNIT, dw[j]);
    }
    __syncthreads();
    for (int k = tid; k < p.K; k += threads) {
        float s = 0.f;
        for (int y = 0; y < (int)blockDim.y; ++y) s += shared[y * p.K + k];
        part[k] = s;
    }
}

// dw[k] = sum of the CTAs' rows, in a fixed order: 32 columns per CTA, its warps share the rows out.  Starts early
// (programmatic launch) and waits for the kernel above.
constexpr int DW_WARPS = 32;
__global__ void __launch_bounds__(DW_WARPS * 32) norm_dw_kernel(const float *parts, int n, int K, float *__restrict__ dw) {
    __shared__ float s[DW_WARPS][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, k = blockIdx.x * 32 + lane;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float sum = 0.f;
    if (k < K) {
#pragma unroll 10
        for (int i = warp; i < n; i += DW_WARPS) sum += parts[(int64_t)i * K + k];
    }
    s[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && k < K) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < DW_WARPS; ++i) t += s[i][lane];
        dw[k] = t;
    }
}
cudaError_t dw_launch(const float *parts, int n, int K, float *dw, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((K + 31) / 32));
    cfg.blockDim = dim3(DW_WARPS * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = n > 0 ? 1 : 0;                        // n = 0: nothing came before it
    return cudaLaunchKernelEx(&cfg, norm_dw_kernel, parts, n, K, dw);
}

constexpr int RING_SMEM = 220 * 1024;        // of an SM, for the CTAs that share it

// A launch of persistent CTAs: at most `most` of them per SM, fewer where a row (stage bytes) would not fit otherwise
struct RowLaunch {
    int ctas, stages, smem;
};
RowLaunch row_launch(int64_t M, const RowShape &s, int most, int stage, int sms) {
    RowLaunch l;
    const int64_t groups = (M + s.rpc - 1) / s.rpc;
    int per_sm = most;
    while (per_sm > 1 && RING_SMEM / per_sm < stage) --per_sm;
    const int fit = RING_SMEM / per_sm / stage;
    l.stages = fit < MAX_STAGES ? fit : MAX_STAGES;
    const int64_t all = (int64_t)sms * per_sm < GEMM_NORM_PARTS ? sms * per_sm : GEMM_NORM_PARTS;
    l.ctas = (int)(groups < all ? groups : all);
    if (groups <= l.ctas) l.stages = 0;      // one row each: straight to registers
    l.smem = l.stages * stage;
    return l;
}
// Raise the kernel's shared-memory limit on the current device, once.
template <auto KERNEL>
cudaError_t allow_smem() {
    static std::mutex mu;
    static bool ready[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[dev]) {
        e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, RING_SMEM);
        ready[dev] = e == cudaSuccess;
    }
    return e;
}

template <typename XT, typename HT, typename YT>
cudaError_t norm_launch(int sms, const NormParams &p, cudaStream_t stream) {
    // Few rows: as many threads as there are units, for the shortest chain.  Many: two units per thread, so that
    // a thread has twice the bytes in flight and half as many warps meet at the barrier (16384 x 4096, bf16 to e4m3: 70.0 us
    // with two, 79.8 with one; 8192 x 2048 without residual: 15.8 and 18.6; at 1024 columns and below the two are equal).
    const int units = p.K / UNIT;
    const RowShape s = row_shape(units, units <= (p.M <= 2 * sms ? 512 : 128) ? 1 : units <= 1024 ? 2 : 4);
    const dim3 block(s.tpr, s.rpc);
    const unsigned ctas = (unsigned)((p.M + s.rpc - 1) / s.rpc);
    if (s.u == 1) norm_kernel<XT, HT, YT, 1><<<ctas, block, 0, stream>>>(p);
    else if (s.u == 2) norm_kernel<XT, HT, YT, 2><<<ctas, block, 0, stream>>>(p);
    else norm_kernel<XT, HT, YT, 4><<<ctas, block, 0, stream>>>(p);
    return cudaGetLastError();
}
template <typename XT, typename HT>
cudaError_t norm_launch(gemm_dtype y, int sms, const NormParams &p, cudaStream_t stream) {
    if (y == GEMM_E4M3) return norm_launch<XT, HT, uint8_t>(sms, p, stream);
    if (y == GEMM_BF16) return norm_launch<XT, HT, __nv_bfloat16>(sms, p, stream);
    return norm_launch<XT, HT, __half>(sms, p, stream);
}
template <typename XT>
cudaError_t norm_launch(gemm_dtype h, gemm_dtype y, int sms, const NormParams &p, cudaStream_t stream) {
    return h == GEMM_F32 ? norm_launch<XT, float>(y, sms, p, stream) : norm_launch<XT, __nv_bfloat16>(y, sms, p, stream);
}

constexpr size_t back_unit(gemm_dtype dy, gemm_dtype h) { return (dy == GEMM_F32 ? 32 : 16) + 2 * (h == GEMM_F32 ? 32 : 16); }

template <typename GT, typename HT, typename YT, int U, int THREADS>
cudaError_t back_launch(const RowShape &s, const RowLaunch &l, NormBackParams p, cudaStream_t stream) {
    const cudaError_t e = allow_smem<norm_back_kernel<GT, HT, YT, U, THREADS>>();
    if (e != cudaSuccess) return e;
    p.stages = l.stages;
    const int joined = s.rpc > 1 ? s.rpc * p.K * (int)sizeof(float) : 0;
    norm_back_kernel<GT, HT, YT, U, THREADS><<<l.ctas, dim3(s.tpr, s.rpc), l.smem > joined ? l.smem : joined, stream>>>(p);
    return cudaGetLastError();
}
template <typename GT, typename HT, typename YT>
cudaError_t back_launch(const RowShape &s, const RowLaunch &l, const NormBackParams &p, cudaStream_t stream) {
    if (s.u == 1) return back_launch<GT, HT, YT, 1, 512>(s, l, p, stream);
    if (s.u == 2) return back_launch<GT, HT, YT, 2, 512>(s, l, p, stream);
    if (s.tpr <= 512) return back_launch<GT, HT, YT, 4, 512>(s, l, p, stream);
    return back_launch<GT, HT, YT, 4, 1024>(s, l, p, stream);
}
template <typename GT, typename HT>
cudaError_t back_launch(gemm_dtype y, const RowShape &s, const RowLaunch &l, const NormBackParams &p, cudaStream_t stream) {
    return y == GEMM_F16 ? back_launch<GT, HT, __half>(s, l, p, stream)
                         : back_launch<GT, HT, __nv_bfloat16>(s, l, p, stream);
}
template <typename GT>
cudaError_t back_launch(gemm_dtype h, gemm_dtype y, const RowShape &s, const RowLaunch &l, const NormBackParams &p,
                        cudaStream_t stream) {
    return h == GEMM_F32 ? back_launch<GT, float>(y, s, l, p, stream)
                         : back_launch<GT, __nv_bfloat16>(y, s, l, p, stream);
}

bool real(gemm_dtype t) { return t == GEMM_F32 || t == GEMM_BF16; }
gemm_status check_sizes(int64_t M, int64_t K) {
    if (M < 0 || K <= 0 || M > INT32_MAX) return GEMM_ERR_INVALID_ARG;
    if (K > MAX_K) return GEMM_ERR_UNSUPPORTED;
    return K % 16 == 0 ? GEMM_OK : GEMM_ERR_ALIGNMENT;
}

}  // namespace
}  // namespace gb300

using namespace gb300;

extern "C" gemm_status gemm_norm_run(int64_t M, int64_t K, gemm_dtype x, gemm_dtype h, gemm_dtype y, float eps,
                                     const void *X, const void *R, const float *W, void *H, void *Y, uint8_t *SFY,
                                     float *RSTD, void *cuda_stream) {
    if (!(eps >= 0.f)) return GEMM_ERR_INVALID_ARG;
    gemm_status st = check_sizes(M, K);
    if (st == GEMM_ERR_INVALID_ARG) return st;
    if (!real(x) || !real(h) || (y != GEMM_E4M3 && y != GEMM_BF16 && y != GEMM_F16)) return GEMM_ERR_UNSUPPORTED;
    if (st != GEMM_OK) return st;
    if (M == 0) return GEMM_OK;
    if (!X || !W || !Y || (y == GEMM_E4M3 && !SFY)) return GEMM_ERR_INVALID_ARG;
    for (const void *p : {X, R, (const void *)W, (const void *)H, (const void *)Y})
        if (!rows::aligned16(p)) return GEMM_ERR_ALIGNMENT;
    int sms = 0;
    st = rows::device_sms(&sms);
    if (st != GEMM_OK) return st;
    const NormParams p{X, R, W, H, Y, SFY, RSTD, M, (int)K, eps};
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(cuda_stream);
    const cudaError_t e = x == GEMM_F32 ? norm_launch<float>(h, y, sms, p, stream)
                                        : norm_launch<__nv_bfloat16>(h, y, sms, p, stream);
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

extern "C" gemm_status gemm_norm_backward(int64_t M, int64_t K, gemm_dtype dy, gemm_dtype h, gemm_dtype y,
                                          const void *DY, const void *DH, const void *H, const float *RSTD,
                                          const float *W, void *DX, float *DW, void *Y, void *workspace,
                                          size_t workspace_bytes, void *cuda_stream) {
    gemm_status st = check_sizes(M, K);
    if (st == GEMM_ERR_INVALID_ARG) return st;
    if (!real(dy) || !real(h) || (Y && y != GEMM_BF16 && y != GEMM_F16)) return GEMM_ERR_UNSUPPORTED;
    if (st != GEMM_OK) return st;
    if (M > 0 && (!DY || !H || !RSTD || !W || !DX)) return GEMM_ERR_INVALID_ARG;
    const int64_t parts_max = M < GEMM_NORM_PARTS ? M : GEMM_NORM_PARTS;
    if (DW && M > 0 && (!workspace || workspace_bytes < (size_t)parts_max * K * sizeof(float))) return GEMM_ERR_INVALID_ARG;
    for (const void *p : {DY, DH, H, (const void *)W, (const void *)DX, (const void *)DW, (const void *)Y,
                          (const void *)workspace})
        if (!rows::aligned16(p)) return GEMM_ERR_ALIGNMENT;
    if (M == 0 && !DW) return GEMM_OK;
    int sms = 0;
    st = rows::device_sms(&sms);
    if (st != GEMM_OK) return st;

    cudaStream_t stream = reinterpret_cast<cudaStream_t>(cuda_stream);
    // Few rows: as many threads as there are units.  Many: two units per thread with everything in registers, 512
    // threads per SM and the ring as deep as fits (4096 x 8192, bf16: 57.2 us; with 64 registers, twice the threads and
    // g and n read again from the ring 67.6; 8192 x 4096: 49.6, one unit per thread 56.1).
    const int units = (int)K / UNIT;
    const RowShape s = row_shape(units, units <= (M <= 3 * sms ? 512 : 128) ? 1 : units <= 1024 ? 2 : 4);
    const int threads = s.tpr * s.rpc, most = s.u == 1 ? 1024 / threads : 512 / threads;
    const RowLaunch l = row_launch(M, s, most < 1 ? 1 : most > 3 ? 3 : most, threads * s.u * (int)back_unit(dy, h), sms);
    const int ctas = l.ctas;
    if (M > 0) {
        // a lone CTA's sums are dw itself
        float *parts = !DW ? nullptr : ctas == 1 ? DW : static_cast<float *>(workspace);
        const NormBackParams p{DY, DH, H, RSTD, W, DX, Y, parts, M, (int)K, 1.f / (float)K, 0};
        const cudaError_t e = dy == GEMM_F32 ? back_launch<float>(h, y, s, l, p, stream)
                                             : back_launch<__nv_bfloat16>(h, y, s, l, p, stream);
        if (e != cudaSuccess) return GEMM_ERR_CUDA;
    }
    if (DW && ctas != 1 && dw_launch(static_cast<const float *>(workspace), ctas, (int)K, DW, stream) != cudaSuccess)
        return GEMM_ERR_CUDA;
    return GEMM_OK;
}
