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

#include "gb300gemm_testing.h"
#include "gemm_rows.cuh"
#include "ptx.cuh"

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
RowShape row_shape(int units, int u, int threads = 256) {      // threads: of a CTA, at least a row's
    RowShape s;
    s.u = u;
    const int need = (units + s.u - 1) / s.u;
    if (need <= 32) {
        s.tpr = 4;
        while (s.tpr < need) s.tpr *= 2;
    } else {
        s.tpr = (need + 31) / 32 * 32;
    }
    s.rpc = s.tpr >= threads ? 1 : threads / s.tpr;
    return s;
}

// Sum over the threads of a row (threadIdx.y), the same in each of them and in a fixed order: within a warp,
// then each warp over the row's warps.  Every thread of the CTA takes part.  `red` holds one float per warp; it may
// be written again after the row's next sum in another place.  OWN: a row's warps wait at a barrier of their own (there
// are fifteen, and at most eight rows of whole warps in a CTA), not for the CTA's other rows.
template <bool OWN>
__device__ __forceinline__ float row_sum(float v, float *red) {
    const int tpr = blockDim.x;
    for (int o = min(tpr, 32) / 2; o > 0; o /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (tpr <= 32) return v;
    const int lane = threadIdx.x & 31, warps = tpr / 32;
    if (lane == 0) red[threadIdx.y * warps + threadIdx.x / 32] = v;
    if (OWN) asm volatile("bar.sync %0, %1;" ::"r"(threadIdx.y + 1), "r"(tpr) : "memory");
    else __syncthreads();
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
// Bound by memory: x and r in, h, y and the scales out, once each.  8192 x 8192, bf16 with residual to e4m3: 71.9 us,
// 6565 GB/s (97% of a copy's rate); with the rows ahead in a ring in shared memory it took longer.  1 x 4096: 1.7 us, a
// launch, a trip to memory and the row's sum.  Without residual and h an element moves half the bytes, and issue slots bound
// it (86%): 32768 x 2048, bf16 to e4m3 52.5 us, 3880 GB/s (57%).
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
    wait_for_previous();
    let_next_launch();
#pragma unroll
    for (int j = 0; j < U; ++j) {
        const int u = threadIdx.x + j * tpr;
        on[j] = row < p.M && u < units;
        load_pieces(x + u * N, on[j], xq[j]);
        load_pieces(r + u * N, on[j] && p.r, rq[j]);
    }
    // w with the row, where registers allow it, or behind the row's sum: with two units only if both inputs are fp32,
    // whose occupancy is no lower for it (4096 x 8192: 66.4 us, 71.4 behind the sum; bf16 x and fp32 h 62.4 and 57.1).
    constexpr bool EARLY_W = U == 1 || (U == 2 && PX + PH == 4);
    float w[U][N];
    if (EARLY_W)
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (on[j]) load(p.w + (threadIdx.x + j * tpr) * N, w[j]);
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
    sum = row_sum<false>(sum, red);
    const float rstd = __frsqrt_rn(sum / (float)p.K + p.eps);
    if (row < p.M && threadIdx.x == 0 && p.rstd) p.rstd[row] = rstd;

#pragma unroll
    for (int j = 0; j < U; ++j) {
        const int u = threadIdx.x + j * tpr;
        if (on[j]) {
            if (!EARLY_W) load(p.w + u * N, w[j]);
#pragma unroll
            for (int i = 0; i < N; ++i) v[j][i] = v[j][i] * rstd * w[j][i];
        }
        if constexpr (sizeof(YT) == 1) {
            const uint32_t code = quantise(v[j], static_cast<uint8_t *>(p.y) + row * p.K + u * N, on[j]);
            if (on[j] && u % (BLOCK / N) == 0) p.sf[row * ((p.K + BLOCK - 1) / BLOCK) + u / (BLOCK / N)] = (uint8_t)code;
        } else if (on[j]) {
            store(static_cast<YT *>(p.y) + row * p.K + u * N, v[j]);
        }
    }
}

// Rows ahead come through a ring in shared memory by asynchronous copies.  Every thread (with fp32, every warp)
// copies the very units that it reads, so the ring needs no barrier of its own.
constexpr int MAX_STAGES = 4;
constexpr int BACK_THREADS = 512;        // w, dw, g and n are 64 registers of each with two units per thread
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Where a piece of a thread's unit lies, in 16-byte places.  Pairs (fp32) lie as in memory, so that a copy's lines stay
// whole, but every other line has them swapped: the same piece of eight threads then comes from all the banks.
template <int PIECES_>
__device__ __forceinline__ int place_of(int thread, int piece) {
    if (PIECES_ == 1) return thread;
    const int at = thread * 2 + piece;
    return at ^ (at >> 3 & 1);
}
// The copies of a warp's units (or of the part of it that has one row, a power of two of lanes): contiguous ones, lane
// by lane.  Calls put(threads from the lane's own, piece).
template <int PIECES_, typename Put>
__device__ __forceinline__ void deal_copies(int tpr, Put put) {
    if constexpr (PIECES_ == 1) {
        put(0, 0);
    } else {
        const int lanes = min(tpr, 32), l = threadIdx.x & (lanes - 1);
#pragma unroll
        for (int i = 0; i < 2; ++i) put((lanes * i + l) / 2 - l, l & 1);
    }
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
    float *parts;        // one row of K per CTA (cluster), or null when dw is not wanted
    int64_t M;
    int K;
    float inverse_k;
    int stages;          // rows of the ring (up to MAX_STAGES), or 0: one row per CTA, loaded where it is used
    int cluster, share;  // CTAs that a row is split over, and the units of each but the last
    int probes;          // SPLIT: the wait's limit
    bool withhold;       // SPLIT: a warp of each cluster keeps its first row's sum to itself (a test)
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Sum over a cluster's threads, the same in each and in a fixed order: every warp's sum goes to every CTA, as one 64-bit
// store of the row's number (from 1) and the value, and who wants the sum looks at the places of its own CTA until all hold
// that row.  (A barrier of the cluster would have the warp's stores to memory wait too: 1.2 us.)
constexpr int MOST_SPLIT = 8, CLUSTER_WARPS = MOST_SPLIT * 16;
constexpr int SUMS = 4;                      // rows whose sums have a place
__device__ __forceinline__ void publish_sum(float v, uint64_t *sums, uint32_t row, int cluster, int rank, bool withhold) {
    for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    const int lane = threadIdx.x & 31, warps = blockDim.x / 32;
    if (lane < cluster && !withhold)
        asm volatile("st.relaxed.cluster.shared::cluster.b64 [%0], %1;" ::"r"(
                         mapa_shared(smem_addr(sums + rank * warps + threadIdx.x / 32), lane)),
                     "l"((uint64_t)row << 32 | __float_as_uint(v))
                     : "memory");
}
// NaN, and with it the rest of the row's gradient, if the others' sums have not come after `probes` looks at a place.  The
// warp then waits for no later row either (`lost`).
constexpr int MOST_PROBES = 1 << 26;         // seconds
__device__ __forceinline__ float published_sum(const uint64_t *sums, uint32_t row, int cluster, int probes, bool &lost) {
    const int places = cluster * (int)(blockDim.x / 32);
    float v = 0.f;
    for (int i = threadIdx.x & 31; i < places; i += 32) {
        uint64_t got;
        for (int left = lost ? 0 : probes;; --left) {
            asm volatile("ld.relaxed.cluster.shared::cta.b64 %0, [%1];" : "=l"(got) : "r"(smem_addr(sums + i)) : "memory");
            if ((uint32_t)(got >> 32) == row) break;
            if (left <= 0) {
                lost = true;
                break;
            }
        }
        v += __uint_as_float((uint32_t)got);
    }
    for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    lost = __any_sync(0xFFFFFFFFu, lost);
    return lost ? __uint_as_float(0x7FC00000u) : v;
}

// A CTA walks rows (rpc at a time) with w and dw in registers; a row costs one barrier, that of its sum.
// Bound by memory: dy, h and dh in, dx (and y) out, once each; then dw's join, 3.5 us that no row's bytes overlap.
// 4096 x 8192, bf16 with y again: 56.9 us, 5895 GB/s (87% of a copy's rate; the rows alone at 97%).  333 x 2064, fp32:
// 7.1 us, two kernels one after the other with a trip to memory each.  Rows of few elements run at a copy's rate, behind
// 5.8 us for the first rows' trip and the last rows' outputs: 16384 x 512, bf16 with y again 20.7 us (18.0 without dw, floor
// 12.4), 65536 x 512 56.9 us (54.4, floor 49.5).
// SPLIT: a row is the work of a cluster, a share of its columns each.  Its sum then takes longer than a row's bytes should, so the
// row before is finished meanwhile, for which dy and h are read from the ring once more.
template <typename GT, typename HT, typename YT, int U, bool SPLIT>
__global__ void __launch_bounds__(BACK_THREADS, U == 1 ? 2 : 1) norm_back_kernel(const __grid_constant__ NormBackParams p) {
    extern __shared__ uint4 ring[];                    // [stages][pieces of a unit: dy, h, dh][U][threads]
    __shared__ float red[2][MAX_WARPS];
    __shared__ uint64_t sums[SUMS][SPLIT ? CLUSTER_WARPS : 1];        // SPLIT: the warps' sums of a row, and its number
    constexpr int PG = PIECES<GT, UNIT>, PH = PIECES<HT, UNIT>, PER_UNIT = PG + 2 * PH;
    const int group = SPLIT ? blockIdx.x / p.cluster : blockIdx.x, groups = SPLIT ? gridDim.x / p.cluster : gridDim.x;
    const int rank = SPLIT ? blockIdx.x - group * p.cluster : 0, first = rank * p.share;       // the CTA's first unit
    const int units = SPLIT ? min(p.share, p.K / UNIT - first) : p.K / UNIT;
    const int tpr = blockDim.x, threads = tpr * blockDim.y, tid = threadIdx.y * tpr + threadIdx.x;
    const uint32_t places = smem_addr(ring);
    const uint32_t unit_bytes = threads * 16, stage_bytes = PER_UNIT * U * unit_bytes;

    const GT *dy = static_cast<const GT *>(p.dy) + first * UNIT;
    const HT *h = static_cast<const HT *>(p.h) + first * UNIT;
    const HT *dh = p.dh ? static_cast<const HT *>(p.dh) + first * UNIT : nullptr;
    const float *weight = p.w + first * UNIT;
    HT *dx = static_cast<HT *>(p.dx) + first * UNIT;
    YT *again = p.y ? static_cast<YT *>(p.y) + first * UNIT : nullptr;
    if (SPLIT) {                               // (the wait is before the loop: no CTA stores into one that has not begun)
        for (int i = tid; i < SUMS * CLUSTER_WARPS; i += threads) (&sums[0][0])[i] = 0;
        __syncwarp();
        cluster_arrive();
    }
    wait_for_previous();
    auto request = [&](int64_t row, int slot) {
        if (PG + PH > 2) __syncwarp();                 // a warp shares its copies: all of it has read what lay there
        if (row < p.M) {
            const uint32_t stage = places + slot * stage_bytes;
            auto copy = [&](auto *from, int first_piece, int j) {
                constexpr int P = PIECES<std::remove_const_t<std::remove_pointer_t<decltype(from)>>, UNIT>;
                deal_copies<P>(tpr, [&](int off, int piece) {
                    const int u = threadIdx.x + off + j * tpr;
                    if (u < units)
                        copy16(stage + (first_piece * U + P * j) * unit_bytes + place_of<P>(tid + off, piece) * 16,
                               from + row * p.K + u * UNIT + piece * 4);
                });
            };
#pragma unroll
            for (int j = 0; j < U; ++j) {
                copy(dy, 0, j);
                copy(h, PG, j);
                if (dh) copy(dh, PG + PH, j);
            }
        }
        copies_commit();
    };
    auto read = [&](auto *from, int64_t row, int slot, int j, int piece, float (&v)[UNIT]) {      // piece: the first of the ring's
        using T = std::remove_const_t<std::remove_pointer_t<decltype(from)>>;
        if (!SPLIT && p.stages == 0) {
            load(from + row * p.K + (threadIdx.x + j * tpr) * UNIT, v);
            return;
        }
        constexpr int P = PIECES<T, UNIT>;
        uint4 q[P];
#pragma unroll
        for (int i = 0; i < P; ++i)
            q[i] = load_shared4(places + slot * stage_bytes + (piece * U + P * j) * unit_bytes + place_of<P>(tid, i) * 16);
        unpack(from, q, v);
    };
    float dw[U][UNIT];
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
        for (int i = 0; i < UNIT; ++i) dw[j][i] = 0.f;

    const int64_t step = (int64_t)groups * blockDim.y;
    const int64_t own = (int64_t)group * blockDim.y + threadIdx.y;      // this thread's first row
    for (int s = 0; s < p.stages; ++s) request(own + s * step, s);
    float w[U][UNIT];
#pragma unroll
    for (int j = 0; j < U; ++j)
        if (threadIdx.x + j * tpr < units) load(weight + (threadIdx.x + j * tpr) * UNIT, w[j]);
    float next_rstd = own < p.M ? p.rstd[own] : 0.f;     // a row ahead, so that no row waits for it
    int slot = 0;
    auto first_pass = [&](int64_t row, int j, float rstd, float (&g)[UNIT], float (&n)[UNIT], float (&sum)[2]) {
        const int u = threadIdx.x + j * tpr;
        read(dy, row, slot, j, 0, g);
        read(h, row, slot, j, PG, n);
#pragma unroll
        for (int i = 0; i < UNIT; ++i) {
            n[i] *= rstd;
            dw[j][i] = fmaf(g[i], n[i], dw[j][i]);
            g[i] *= w[j][i];
            sum[i & 1] = fmaf(g[i], n[i], sum[i & 1]);
        }
        if (again) {
            float y[UNIT];
#pragma unroll
            for (int i = 0; i < UNIT; ++i) y[i] = n[i] * w[j][i];
            store(again + row * p.K + u * UNIT, y);
        }
    };
    auto second_pass = [&](int64_t row, int at, int j, float rstd, float c, const float (&g)[UNIT], const float (&n)[UNIT]) {
        float d[UNIT];
        if (dh) {
            read(dh, row, at, j, PG + PH, d);
        } else {
#pragma unroll
            for (int i = 0; i < UNIT; ++i) d[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < UNIT; ++i) d[i] += rstd * (g[i] - n[i] * c);
        store(dx + row * p.K + (threadIdx.x + j * tpr) * UNIT, d);
    };
    if constexpr (SPLIT) {
        cluster_wait();
        float rstd_before = 0.f;
        int before = 0;                                              // the slot of the row before
        uint32_t turn = 0;                                           // the cluster's rows before this one
        bool lost = false;
        for (int64_t row = own; row - step < p.M; row += step) {
            const float rstd = next_rstd;
            next_rstd = row + step < p.M ? p.rstd[row + step] : 0.f;
            if (row < p.M) {                                         // (the same in the whole cluster)
                wait_stage(p.stages - 1);
                if (PG + PH > 2) __syncwarp();
                float sum[2] = {0.f, 0.f};
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    float g[UNIT], n[UNIT];
                    if (threadIdx.x + j * tpr < units) first_pass(row, j, rstd, g, n, sum);
                }
                publish_sum(sum[0] + sum[1], sums[turn % SUMS], turn + 1, p.cluster, rank,
                            p.withhold && turn == 0 && rank == 0 && threadIdx.x < 32);
            } else {                                                 // (once, behind the last row)
                // No CTA's shared memory goes while another may still store into it, as one may that had given up waiting:
                // the wait is before the kernel's end.  (Behind the last row's outputs the few rows of a small call would
                // wait for those: 8 x 16384, bf16 7.6 us, 7.3 here.)
                cluster_arrive();
            }
            if (row != own) {
                // A place is written again four rows on, for which its writer has every warp's sum of the second row on,
                // sent behind this read.  (A writer that has stopped waiting may be earlier: this wait then runs out too.)
                const float c = published_sum(sums[(turn - 1) % SUMS], turn, p.cluster, p.probes, lost) * p.inverse_k;
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    if (threadIdx.x + j * tpr >= units) continue;
                    float g[UNIT], n[UNIT];
                    read(dy, row - step, before, j, 0, g);
                    read(h, row - step, before, j, PG, n);
#pragma unroll
                    for (int i = 0; i < UNIT; ++i) {
                        n[i] *= rstd_before;
                        g[i] *= w[j][i];
                    }
                    second_pass(row - step, before, j, rstd_before, c, g, n);
                }
                request(row + (p.stages - 1) * step, before);        // the thread itself has read what lay there
            }
            rstd_before = rstd;
            before = slot;
            slot = slot + 1 == p.stages ? 0 : slot + 1;
            ++turn;
        }
    } else {
        int turn = 0;
        for (int64_t row = own; row - threadIdx.y < p.M; row += step, turn ^= 1) {
            const bool live = row < p.M;
            const float rstd = next_rstd;
            next_rstd = row + step < p.M ? p.rstd[row + step] : 0.f;
            if (p.stages) {
                wait_stage(p.stages);
                if (PG + PH > 2) __syncwarp();
            }
            float g[U][UNIT], n[U][UNIT], sum[2] = {0.f, 0.f};
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (live && threadIdx.x + j * tpr < units) first_pass(row, j, rstd, g[j], n[j], sum);
            const float c = row_sum<true>(sum[0] + sum[1], red[turn]) * p.inverse_k;
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (live && threadIdx.x + j * tpr < units) second_pass(row, slot, j, rstd, c, g[j], n[j]);
            if (p.stages) request(row + p.stages * step, slot);          // the thread itself has read what lay there
            slot = slot + 1 >= p.stages ? 0 : slot + 1;
        }
    }
    let_next_launch();

    // the CTA's sums in a fixed order: rows of threads first, then (norm_dw_kernel) CTAs
    float *part = p.parts + (int64_t)group * p.K + first * UNIT;
    if (p.parts && (SPLIT || blockDim.y == 1)) {
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int u = threadIdx.x + j * tpr;
            if (u < units) store(part + u * UNIT, dw[j]);
        }
    }
    if (SPLIT) {
        __syncwarp();
        cluster_wait();
    }
    if (SPLIT || !p.parts || blockDim.y == 1) return;
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

// dw[k] = sum of the CTAs' rows, in a fixed order: COLUMNS columns per CTA, its warps share the rows out, 32 / COLUMNS of
// them at a time.  Few columns for small K and many rows, so that all SMs take part: 1000 x 2048, bf16 9.9 us
// with eight columns, 11.2 with 32 (`spread`; 333 x 2064, fp32, a row per CTA: 7.5 and 7.1).
constexpr int DW_WARPS = 32;
template <int COLUMNS>
__global__ void __launch_bounds__(DW_WARPS * 32) norm_dw_kernel(const float *parts, int n, int K, float *__restrict__ dw) {
    constexpr int ROWS = 32 / COLUMNS;
    __shared__ float s[DW_WARPS][COLUMNS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, c = lane % COLUMNS, k = blockIdx.x * COLUMNS + c;
    wait_for_previous();
    let_next_launch();
    float sum = 0.f;
    if (k < K) {
#pragma unroll 10
        for (int i = warp * ROWS + lane / COLUMNS; i < n; i += DW_WARPS * ROWS) sum += parts[(int64_t)i * K + k];
    }
#pragma unroll
    for (int o = COLUMNS; o < 32; o *= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane < COLUMNS) s[warp][c] = sum;
    __syncthreads();
    if (warp != 0) return;
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < DW_WARPS; i += ROWS) t += s[i + lane / COLUMNS][c];
#pragma unroll
    for (int o = COLUMNS; o < 32; o *= 2) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    if (lane < COLUMNS && k < K) dw[k] = t;
}
cudaError_t dw_launch(const float *parts, int n, int K, float *dw, int sms, bool spread, cudaStream_t stream) {
    const int at_once = spread ? 2 * sms : 0;            // CTAs
    if (K <= 8 * at_once) return launch(norm_dw_kernel<8>, (K + 7) / 8, DW_WARPS * 32, 0, stream, parts, n, K, dw);
    if (K <= 16 * at_once) return launch(norm_dw_kernel<16>, (K + 15) / 16, DW_WARPS * 32, 0, stream, parts, n, K, dw);
    return launch(norm_dw_kernel<32>, (K + 31) / 32, DW_WARPS * 32, 0, stream, parts, n, K, dw);
}

constexpr int RING_SMEM = 220 * 1024;        // of an SM, for the CTAs that share it

// A launch of persistent CTAs: at most `most` of them per SM, fewer where a row (stage bytes) would not fit otherwise
struct RowLaunch {
    int groups, stages, smem;                // groups: CTAs, or clusters of them
};
RowLaunch row_launch(int64_t M, int rpc, int most, int stage, int resident, bool split) {
    RowLaunch l;
    const int64_t groups = (M + rpc - 1) / rpc;
    int per_sm = most;
    while (per_sm > 1 && RING_SMEM / per_sm < stage) --per_sm;
    const int fit = RING_SMEM / per_sm / stage;
    l.stages = fit < MAX_STAGES ? fit : MAX_STAGES;
    const int64_t all = (int64_t)resident * per_sm < GEMM_NORM_PARTS ? resident * per_sm : GEMM_NORM_PARTS;
    l.groups = (int)(groups < all ? groups : all);
    if (groups <= l.groups && !split) l.stages = 0;      // one row each: straight to registers
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
    // with two, 79.8 with one; bf16 to e4m3 without residual at 8192 x 2048: 15.4 and 18.3; at 1024 columns and below the two
    // are equal).
    const int units = p.K / UNIT;
    const RowShape s = row_shape(units, units <= (p.M <= 2 * sms ? 512 : 128) ? 1 : units <= 1024 ? 2 : 4);
    const dim3 block(s.tpr, s.rpc);
    const int ctas = (int)((p.M + s.rpc - 1) / s.rpc);
    if (s.u == 1) return launch(norm_kernel<XT, HT, YT, 1>, ctas, block, 0, stream, p);
    if (s.u == 2) return launch(norm_kernel<XT, HT, YT, 2>, ctas, block, 0, stream, p);
    return launch(norm_kernel<XT, HT, YT, 4>, ctas, block, 0, stream, p);
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

// The next calls' limit of the wait for a split row's sums, and whether one is withheld (gemm_testing_set_norm_fault)
thread_local int probes = MOST_PROBES;
thread_local bool withhold = false;

// How many clusters of `cluster` CTAs run at once, each CTA with an SM's shared memory to itself
template <auto KERNEL>
cudaError_t resident_clusters(int cluster, int *out) {
    static std::mutex mu;
    static int known[64][MOST_SPLIT + 1];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    int &n = known[dev][cluster];
    if (n == 0) {
        const Launch l(cluster, BACK_THREADS, RING_SMEM, cluster, nullptr, false);
        e = cudaOccupancyMaxActiveClusters(&n, KERNEL, &l.config);
        if (e == cudaSuccess && n <= 0) e = cudaErrorInvalidConfiguration;
    }
    *out = n;
    return e;
}

// A unit of a row in the ring: dy, h, dh
template <typename GT, typename HT>
constexpr int UNIT_BYTES = (PIECES<GT, UNIT> + 2 * PIECES<HT, UNIT>) * 16;
// How the rows are spread: over threads, and over a cluster's CTAs from `share` units on
struct BackShape {
    RowShape s;
    int cluster, share;
};
// Few rows (up to three per SM): as many threads as there are units (333 x 1536, bf16 4.8 us, 6.3 with two units each;
// 1000 x 2048 11.7 and 9.8).  Many: two units per thread with everything in registers, 512 threads
// per SM and the ring as deep as fits (4096 x 8192, bf16: 56.9 us; with 64 registers, twice the threads and g and n
// read again from the ring 67.6).
// Rows of more than 8192 elements, and those of which an SM's shared memory does not hold three, are split over 2, 4 or
// 8 CTAs.  2048 x 16384, bf16: 59.4 us with two CTAs per row; by one CTA with four units per thread, and w read again
// for every row, 88.3.  4096 x 8192, all fp32: 94.1 us with two, 106.6 with one and a ring of two rows.
constexpr int LINE = 16;                     // units of 256 bytes
BackShape back_shape(int64_t M, int K, int sms, int unit_bytes) {
    const int units = K / UNIT;
    BackShape b;
    b.cluster = 1;
    while (units > b.cluster * 2 * BACK_THREADS) b.cluster *= 2;
    for (;; b.cluster *= 2) {
        if (b.cluster == 1) {
            b.share = units;
            b.s = row_shape(units, units <= (M <= 3 * sms ? BACK_THREADS : 128) ? 1 : 2);
            // With several rows for every CTA, large CTAs, of which there are fewer partial sums of dw: 16384 x 1024, bf16
            // 33.9 us, 41.5 with CTAs of 256 threads.
            const RowShape large = row_shape(units, b.s.u, BACK_THREADS);
            const int row = large.tpr * large.rpc * large.u * unit_bytes;
            if (M >= (int64_t)4 * sms * large.rpc && row * 3 * (large.u == 1 ? 2 : 1) <= RING_SMEM) b.s = large;
        } else {
            b.share = (units + LINE * b.cluster - 1) / (LINE * b.cluster) * LINE;        // whole lines of memory
            b.s = row_shape(b.share, 2);
            b.s.rpc = 1;
        }
        if (b.s.u == 1 || b.s.tpr * b.s.rpc * 2 * unit_bytes * 3 <= RING_SMEM) return b;
    }
}

// `parts`: how many rows of partial sums there are
template <typename GT, typename HT, typename YT, int U, bool SPLIT>
cudaError_t back_launch(const BackShape &b, NormBackParams p, float *dw, int sms, int *parts, cudaStream_t stream) {
    constexpr auto KERNEL = norm_back_kernel<GT, HT, YT, U, SPLIT>;
    cudaError_t e = allow_smem<KERNEL>();
    int resident = sms;
    if (e == cudaSuccess && SPLIT) e = resident_clusters<KERNEL>(b.cluster, &resident);
    if (e != cudaSuccess) return e;
    const int threads = b.s.tpr * b.s.rpc, most = SPLIT ? 1 : U == 1 ? 1024 / threads : BACK_THREADS / threads;
    const RowLaunch l = row_launch(p.M, b.s.rpc, most < 1 ? 1 : most > 3 ? 3 : most, threads * U * UNIT_BYTES<GT, HT>,
                                   resident, SPLIT);
    p.stages = l.stages;
    p.cluster = b.cluster;
    p.share = b.share;
    if (dw && l.groups == 1) p.parts = dw;               // a lone group's sums are dw itself
    *parts = l.groups;
    const int joined = b.s.rpc > 1 ? b.s.rpc * p.K * (int)sizeof(float) : 0;
    const Launch run(l.groups * b.cluster, dim3(b.s.tpr, b.s.rpc), l.smem > joined ? l.smem : joined, b.cluster, stream);
    return cudaLaunchKernelEx(&run.config, KERNEL, p);
}
template <typename GT, typename HT, typename YT>
cudaError_t back_launch(const NormBackParams &p, float *dw, int sms, int *parts, cudaStream_t stream) {
    const BackShape b = back_shape(p.M, p.K, sms, UNIT_BYTES<GT, HT>);
    if (b.cluster > 1) return back_launch<GT, HT, YT, 2, true>(b, p, dw, sms, parts, stream);
    if (b.s.u == 1) return back_launch<GT, HT, YT, 1, false>(b, p, dw, sms, parts, stream);
    return back_launch<GT, HT, YT, 2, false>(b, p, dw, sms, parts, stream);
}
template <typename GT, typename HT>
cudaError_t back_launch(gemm_dtype y, const NormBackParams &p, float *dw, int sms, int *parts, cudaStream_t stream) {
    return y == GEMM_F16 ? back_launch<GT, HT, __half>(p, dw, sms, parts, stream)
                         : back_launch<GT, HT, __nv_bfloat16>(p, dw, sms, parts, stream);
}
template <typename GT>
cudaError_t back_launch(gemm_dtype h, gemm_dtype y, const NormBackParams &p, float *dw, int sms, int *parts, cudaStream_t stream) {
    return h == GEMM_F32 ? back_launch<GT, float>(y, p, dw, sms, parts, stream)
                         : back_launch<GT, __nv_bfloat16>(y, p, dw, sms, parts, stream);
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
    int parts = 0;
    if (M > 0) {
        const NormBackParams p{DY, DH, H, RSTD, W, DX, Y, DW ? static_cast<float *>(workspace) : nullptr, M, (int)K,
                               1.f / (float)K, 0, 1, 0, probes, withhold};
        const cudaError_t e = dy == GEMM_F32 ? back_launch<float>(h, y, p, DW, sms, &parts, stream)
                                             : back_launch<__nv_bfloat16>(h, y, p, DW, sms, &parts, stream);
        if (e != cudaSuccess) return GEMM_ERR_CUDA;
    }
    if (DW && parts != 1 && dw_launch(static_cast<const float *>(workspace), parts, (int)K, DW, sms, M > parts, stream) != cudaSuccess)
        return GEMM_ERR_CUDA;
    return GEMM_OK;
}

// Test hook (declared in include/gb300gemm_testing.h): split rows' waits that run out.
extern "C" gemm_status gemm_testing_set_norm_fault(int limit) {
    if (limit < 0) return GEMM_ERR_INVALID_ARG;
    probes = limit ? limit : MOST_PROBES;
    withhold = limit != 0;
    return GEMM_OK;
}
