// The first product of a feed-forward block with its gated unit in one kernel, and the product
// that enters the unit from behind with the unit's gradient (gemm_gated_run, gemm_gated_back_run
// in include/gb300gemm.h):
//
//   forward    z = X·[Wg; Wu]ᵀ = [g | u],  a = g / (1 + exp(-g)) * u,  g and u kept in 8 bits
//   backward   da = DY·W2,  [dg | du] from da and the kept g, u,  a again
//
// The roles are those of gemm_tc_kernel (gemm_kernel.cuh): a TMA producer warp, a warp with the
// MMA issuing thread, scale-copying warps for block-scaled operands, epilogue warps.  What differs
// is what a tile is and what its epilogue does:
//
//   * Forward: 64 columns of A take 128 columns of the product, 64 of g and then the same 64 of u.  The
//     weights are mapped as [2][F][K], so that a box of 64 rows of either half is zero past F.
//     Both accumulators of an element are then in the same lane of tensor memory, 64 columns apart:
//     the unit needs no exchange between threads.  A CTA pair's tile has 128 columns of A, 64 in
//     each CTA's half of the MMA's N.
//   * Where a pair's last round of tiles would leave half of the pairs or more without work, its tiles are
//     halved: 64 columns of A, the leader holding g's rows and its peer u's (backward: 128 columns).
//   * Block scales are packed by a kernel before (gemm_sfpack.cu) and come by TMA, as in gemm_tc_kernel, or
//     (GROUPED: single CTAs, whose products are short, where every row of scales begins at a multiple of 16 bytes) are
//     read as the operands' owners have them: the copying warp loads sixteen bytes of a row (a group of four
//     k-blocks) ahead of their use, writes the group's words to shared memory in tensor memory's order and copies them
//     there, into a ring of groups of its own: 64 x 8192 x 4096 takes 17.4 us, 22.6 with the packing kernel (captured 17.7
//     and 20.3).  (For pairs the way over both CTAs' warps takes 2 us per group, twice its MMAs' time: 4096 x 8192 x 8192 458 us,
//     385 with the packing kernel; rows that begin anywhere cost ten loads for one, 30 us at 64 x 8192 x 4064; a second form for
//     rows at multiples of 8 bytes in the same kernel costs the first one 2.5 us.)
//   * A thread owns a row; its chunk of 32 columns is one scale block of e4m3, so that a block's
//     maximum is a thread's own.
//   * Backward: B is N-contiguous (W2 as the forward product has it), g and u come as 8-bit codes
//     straight from memory, one chunk ahead of their use, and dz and a leave through TMA boxes.  (A tile ahead, or brought to L2
//     a tile ahead: no faster.  4096 x 8192 x 2048 takes 114 us, the product alone 87; the traffic of the codes and that of dz
//     are 11 to 12 us of the rest each, the arithmetic 1.5.)
//   * Two warps may issue a CTA's MMAs, every other k-block each, into accumulators that the epilogue adds: one thread takes 450
//     clocks for a k-block's four MMAs, their wait and their commit, whatever their N.  Backward tiles of 64 columns: 0.158 us per
//     k-block, 0.237 with one.  Tiles of 128: forward 512 x 2048 x 2048 9.8 us, 10.8, backward 1024 x 2048 x 1024 9.4, 9.9; sliced
//     ones, whose operands' way from L2 takes as long, 128 x 4096 x 4096 17.8, 17.5 with one.
//   * Where tiles are few, a tile's K is cut into slices over the single CTAs of a cluster, which exchange their sums
//     before the unit: each finishes the share of the tile's 32 x 32 pieces that it owns, adding all slices in their order.
// Every wait is bounded as in gemm_tc_kernel.
#pragma once

#include "gemm_kernel.cuh"
#include "gemm_rows.cuh"

namespace gb300 {

// Compile-time shape of one kernel instance: HN columns of A per tile; the rest as in TileCfg.
template <int CG_, int KIND_, bool BACK_, int HN_, int STAGES_, int ACC_BUFS_, int EPI_WARPS_, int COPIERS_ = 0,
          bool GROUPED_ = false, bool SLICED_ = false, int ISSUERS_ = 1>
struct GatedCfg {
    static constexpr int CG = CG_;
    static constexpr int KIND = KIND_;
    static constexpr bool SCALED = KIND != KIND_F16;
    static constexpr bool BACK = BACK_;
    static constexpr int HN = HN_;
    static constexpr int BN = BACK ? HN : 2 * HN;               // columns of the MMA
    // the narrow form of a tile: all that a single CTA has, a pair's halved tile
    static constexpr int NARROW = HN / CG_;                     // columns of A
    static_assert(BACK || NARROW == 64, "64 columns of g and of u");
    static constexpr int STAGES = STAGES_;
    static constexpr int ACC_BUFS = ACC_BUFS_;
    static constexpr int EPI_WARPS = EPI_WARPS_;
    static constexpr int COPIERS = COPIERS_;
    static constexpr bool COPIER = COPIERS > 0;
    static constexpr int COPY_WARP = 2 + EPI_WARPS;
    // warps that issue MMAs, each every ISSUERS-th k-block into an accumulator of its own
    static constexpr int ISSUERS = ISSUERS_;
    static constexpr int SECOND_ISSUER = COPY_WARP + COPIERS;   // the first one is warp 1
    static constexpr int THREADS = 32 * (SECOND_ISSUER + ISSUERS - 1);
    static_assert(ISSUERS == 1 || (ISSUERS == 2 && CG == 1), "one or, in single CTAs, two");
    // The barriers of loaded stages: an even number with two issuers, so that each has its own, whose phases it sees one after
    // the other (a wait for one phase says nothing where the phase before it may be open)
    static constexpr int FULLS = STAGES_ % ISSUERS == 0 ? STAGES_ : 2 * STAGES_;
    static_assert(EPI_WARPS == 8, "two epilogue warps per TMEM lane window");
    // chunks of A's columns one epilogue warp handles
    static constexpr int WCHUNKS = HN / 2 / EPI_COLS, NARROW_WCHUNKS = NARROW / 2 / EPI_COLS;
    static constexpr int ELEM_BITS = KIND == KIND_F16 ? 16 : 8;
    static constexpr int ELEM_BYTES = ELEM_BITS / 8;
    static constexpr int BK = 1024 / ELEM_BITS;                 // K elements per stage: one 128-byte row
    static constexpr int MMA_K = 256 / ELEM_BITS;
    static constexpr int ATOM_MN = 1024 / ELEM_BITS;            // N elements of an N-contiguous operand's atom
    static constexpr int ATOM_BYTES = BK * 128;
    static constexpr int A_BYTES = TILE_M * 128;
    static constexpr int B_ROWS = BN / CG;                      // B rows held by one CTA
    static constexpr int B_BYTES = B_ROWS * 128;
    static constexpr int SF_WORDS = SCALED ? BK / 32 / 4 : 0;
    static constexpr int SF_PER_MMA = 1;
    static constexpr int HALVES = (BN + 127) / 128;
    static constexpr int SFA_BYTES = 512 * SF_WORDS;
    static constexpr int SFB_BYTES = 512 * SF_WORDS * HALVES;
    static constexpr int BOX_BYTES = 64 * 128;                  // a box of B: 64 rows (backward: columns) of 128 bytes
    static constexpr int BOXES = B_BYTES / BOX_BYTES;
    static constexpr int NARROW_BOXES = (BACK ? NARROW : 2 * NARROW) / CG / 64;
    static constexpr int TX_AB = CG * (A_BYTES + B_BYTES);
    static constexpr int NARROW_TX_AB = CG * (A_BYTES + NARROW_BOXES * BOX_BYTES);
    static constexpr bool GROUPED = GROUPED_;                   // the copying warp packs the scales
    static constexpr bool PACKED = SCALED && !GROUPED;          // they come packed, a stage's with its operands
    static_assert(!GROUPED || (SCALED && CG == 1), "scales packed by a single CTA");
    static constexpr int TX_SF = CG * (SFA_BYTES + SFB_BYTES);
    static constexpr int NARROW_TX_SF = CG * (SFA_BYTES + 512 * SF_WORDS);
    static constexpr int SF_GROUP = PACKED ? 1 : 4;             // k-blocks of a group of scales
    static constexpr int SF_RING = PACKED ? STAGES : GROUPED ? 4 : 0;   // groups in shared and in tensor memory
    static constexpr int SF_BLOCKS = SF_WORDS * (1 + HALVES);   // 512-byte blocks of scales of a stage: X's, W's
    // an epilogue warp's staging: 32 rows of a chunk of each output (16-bit: 2 KiB, 8-bit: 1 KiB)
    static constexpr int EPI_BUF = BACK ? 3 * 2048 : 2048 + 2 * 1024;
    static constexpr int align1k(int x) { return (x + 1023) / 1024 * 1024; }
    static constexpr int OFF_A = 0;
    static constexpr int OFF_B = OFF_A + STAGES * A_BYTES;
    static constexpr int OFF_SF = OFF_B + STAGES * B_BYTES;
    static constexpr int OFF_EPI = align1k(OFF_SF + SF_RING * SF_GROUP * SF_BLOCKS * 512);
    // Tiles sliced along K over a cluster's CTAs (2, 4 or 8): of the tile's eight pieces, a warp's 32 rows and half of the tile's
    // columns, a CTA owns 8 / slices.  Each has a staging buffer, and behind those the other slices' fp32 sums of it.
    static constexpr bool SLICED = SLICED_;
    static_assert(!SLICED || CG == 1, "slices over single CTAs");
    static constexpr int MAX_SLICES = SLICED ? 8 : 1;
    static constexpr int PIECE = 4096 * WCHUNKS * (BACK ? 1 : 2);
    static constexpr int larger(int x, int y) { return x > y ? x : y; }
    static constexpr int EPI_BYTES = SLICED ? larger(EPI_BUF + 7 * PIECE, larger(2 * (EPI_BUF + 3 * PIECE), 4 * (EPI_BUF + PIECE)))
                                            : EPI_WARPS * EPI_BUF;
    static constexpr int OFF_BAR = OFF_EPI + EPI_BYTES;
    // full[FULLS], empty[STAGES], tfull[2], tempty[2], drain, then with COPIER: cdrain and, per group of scales,
    // sffull (packed ones have landed), sfready (grouped ones are in tensor memory), sfempty (their MMAs are done)
    // and last, with slices, recv[4] (the other slices' sums of an owned piece have landed)
    static constexpr int NBAR = FULLS + STAGES + 5 + (COPIER ? 3 * SF_RING + 1 : 0) + (SLICED ? 4 : 0);
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;         // tmem base slot, abort flag
    static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;     // + alignment slack
    static constexpr int SF_SLOT = 4 * SF_WORDS * (1 + HALVES);
    static constexpr int ACC_COLS = ISSUERS * BN;               // of an accumulator buffer
    static constexpr int SF_COL0 = ACC_BUFS * ACC_COLS;
    static_assert(CG == 1 || CG == 2, "CTA group");
    static_assert(KIND == KIND_F16 || KIND == KIND_MXF8, "operand kind");
    static_assert(!BACK || KIND == KIND_F16, "the backward product has 16-bit operands");
    static_assert(COPIER == SCALED, "block-scaled instances have copier warps");
    static_assert(SF_COL0 + SF_RING * SF_GROUP * SF_SLOT <= 512, "TMEM budget");
    static_assert(SMEM_BYTES <= 232448, "shared-memory budget");
    static_assert(A_BYTES % 1024 == 0 && B_BYTES % 1024 == 0 && EPI_BUF % 1024 == 0, "1024-byte regions");
    static_assert(BN <= 256 && SF_WORDS <= 1, "tile columns, one word of scales per stage and row");
    static_assert(ACC_BUFS == 1 || ACC_BUFS == 2, "accumulator buffers");
};

// A unit of work: rows [128 CG tm, ...) and HN columns of A from f0, or NARROW of them.  The first `whole` units are
// tiles; the tiles behind them come as two halves each.
struct GatedUnit {
    int tm, f0;
    bool narrow;
};
template <class Cfg>
__device__ __forceinline__ GatedUnit gated_unit(const GatedParams &p, int u) {
    const bool half = Cfg::CG == 2 && u >= p.whole;
    const int t = half ? p.whole + (u - p.whole) / 2 : u;
    GatedUnit w;
    int tn;
    tile_coords(t, p.tiles_m, p.group_m, w.tm, tn, p.tiles_n);
    w.f0 = tn * Cfg::HN + (half ? ((u - p.whole) & 1) * Cfg::NARROW : 0);
    w.narrow = Cfg::CG == 1 || half;
    return w;
}

// k-block kb is the first of its group in the order in which a unit of this round walks K
template <class Cfg>
__device__ __forceinline__ bool group_begins(int kb, uint32_t round) {
    const int edge = GB300_SERPENTINE_K && (round & 1u) ? Cfg::SF_GROUP - 1 : 0;
    return kb % Cfg::SF_GROUP == edge;
}

// 32 values of a row quantised as one scale block: codes to shared memory (32-byte row `lane` of a
// 32-byte-swizzled box), the block's scale code returned
__device__ __forceinline__ uint32_t quantise_chunk(const float (&v)[32], uint32_t box, int lane) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) amax = fmaxf(amax, fabsf(v[i]));      // fmaxf drops NaN
    const uint32_t code = rows::scale_code(amax);
    const float2 inv = rows::both(rows::scale_inverse(code));
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float *x = v + 16 * c + 4 * i;
            const float2 a = rows::mul2(make_float2(x[0], x[1]), inv), b = rows::mul2(make_float2(x[2], x[3]), inv);
            w[i] = rows::e4m3x2(a.x, a.y) | rows::e4m3x2(b.x, b.y) << 16;
        }
        st_shared_v4(box + swz_off<32>(lane, c), w[0], w[1], w[2], w[3]);
    }
    return code;
}

// 32 values of a row rounded to 16 bits: 64-byte row `lane` of a 64-byte-swizzled box
__device__ __forceinline__ void round_chunk(const float (&v)[32], bool bf16, uint32_t box, int lane) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const uint4 q = bf16 ? rows::pack8(static_cast<const __nv_bfloat16 *>(nullptr), v + 8 * c)
                             : rows::pack8(static_cast<const __half *>(nullptr), v + 8 * c);
        st_shared_v4(box + swz_off<64>(lane, c), q.x, q.y, q.z, q.w);
    }
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS, 1)
    gated_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                 const __grid_constant__ CUtensorMap tmSFX, const __grid_constant__ CUtensorMap tmSFW,
                 const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmZ,
                 const GatedParams p) {
    constexpr int CG = Cfg::CG;
    constexpr int STAGES = Cfg::STAGES;
    constexpr int BN = Cfg::BN;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;

    uint64_t *full = reinterpret_cast<uint64_t *>(smem + Cfg::OFF_BAR);
    uint64_t *empty = full + Cfg::FULLS;
    uint64_t *tfull = empty + STAGES;
    uint64_t *tempty = tfull + 2;
    uint64_t *drain = tempty + 2;
    uint64_t *cdrain = drain + 1;                         // COPIER only
    uint64_t *sffull = cdrain + 1;                        // COPIER only, as the next two
    uint64_t *sfready = sffull + Cfg::SF_RING;
    uint64_t *sfempty = sfready + Cfg::SF_RING;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Cfg::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + Cfg::OFF_MISC + 4);
    const Waiter W{abort_flag, p.status, p.timeout_ns};
    uint64_t *recv = full + Cfg::NBAR - 4;                // SLICED only
    // a tile's slice of K: k-blocks [kb0, kb1)
    const int slices = Cfg::SLICED ? p.slices : 1, slice = Cfg::SLICED ? (int)cluster_ctarank() : 0;
    const int kb0 = (int)((int64_t)slice * p.num_kb / slices), kb1 = (int)((int64_t)(slice + 1) * p.num_kb / slices);

    if (threadIdx.x == 0) {
        prefetch_tensormap(&tmX);
        prefetch_tensormap(&tmW);
        if constexpr (Cfg::PACKED) {
            prefetch_tensormap(&tmSFX);
            prefetch_tensormap(&tmSFW);
        }
        if (p.has_a) prefetch_tensormap(&tmA);
        if (p.has_z) prefetch_tensormap(&tmZ);
        // the producer's arrival and, with packed scales, each copier warp's commit
        for (int s = 0; s < Cfg::FULLS; ++s) mbar_init(&full[s], 1 + (Cfg::PACKED ? Cfg::COPIERS : 0));
        for (int s = 0; s < STAGES; ++s) mbar_init(&empty[s], 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], Cfg::ISSUERS);
            mbar_init(&tempty[b], Cfg::EPI_WARPS * CG);
        }
        mbar_init(drain, Cfg::ISSUERS);
        if constexpr (Cfg::COPIER) {
            for (int i = 0; i < Cfg::SF_RING; ++i) {
                mbar_init(&sffull[i], 1);
                mbar_init(&sfready[i], 1);
                mbar_init(&sfempty[i], Cfg::ISSUERS);
            }
            mbar_init(cdrain, Cfg::COPIERS);
        }
        if constexpr (Cfg::SLICED)
            for (int i = 0; i < 4; ++i) mbar_init(&recv[i], 1);
        *abort_flag = 0;
        fence_mbarrier_init();
    }
    if (warp == 1) {
        tmem_alloc<CG>(smem_addr(tmem_slot), 512);
        tmem_relinquish<CG>();
    }
    tc_fence_before_sync();
    if constexpr (CG == 2 || Cfg::SLICED) cluster_sync(); else __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    rows::wait_for_previous();
    rows::let_next_launch();

    // (sliced tiles all run at once: a cluster has one)
    const int unit0 = (int)blockIdx.x / (CG * slices);
    const int unit_step = (int)gridDim.x / (CG * slices);

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            int s = 0, fs = 0;
            uint32_t ph = 0, round = 0;
            bool ok = true;
            for (int n = unit0; ok && n < p.units; n += unit_step, ++round) {
                const GatedUnit w = gated_unit<Cfg>(p, n);
                const int m0 = (w.tm * CG + (int)rank) * TILE_M;
                for (int j = 0; j < kb1 - kb0; ++j) {
                    const int kb = kb_at(j, kb0, kb1, round);
                    if (!W.wait(&empty[s], ph ^ 1u)) { ok = false; break; }
                    const bool withhold = p.fault == 1 && round == 0 && j == 0;
                    const uint32_t fb = smem_addr(&full[fs]);
                    const uint32_t bar = CG == 1 ? fb : mapa_shared(fb, 0);      // the leader's
                    if constexpr (Cfg::PACKED) {          // the scales first: the copier warps start on them
                        if (rank == 0) mbar_arrive_expect_tx(&sffull[s], w.narrow ? Cfg::NARROW_TX_SF : Cfg::TX_SF);
                        const uint32_t sb = smem_addr(&sffull[s]);
                        const uint32_t sbar = CG == 1 ? sb : mapa_shared(sb, 0);
                        auto load_sf = [&](uint32_t to, const CUtensorMap *m, int row) {
                            if constexpr (CG == 1) tma_load_2d(to, m, sbar, 0, row);
                            else tma_load_2d_pair(to, m, sbar, 0, row);
                        };
                        const uint32_t dst = smem_addr(smem + Cfg::OFF_SF + s * Cfg::SF_BLOCKS * 512);
                        // 512-byte blocks, four rows of the packed scales: one per (128 rows of X, k-block) and
                        // per (64 columns of A, k-block)
                        load_sf(dst, &tmSFX, checked_y(p.status, ((w.tm * CG + (int)rank) * p.num_kb + kb) * 4,
                                                       p.tiles_m * CG * p.num_kb * 4));
#pragma unroll
                        for (int i = 0; i < Cfg::HALVES; ++i)
                            if (i == 0 || !w.narrow)      // (HALVES is 1 in a single CTA)
                                load_sf(dst + 512 * (1 + i), &tmSFW,
                                        checked_y(p.status, ((w.f0 / 64 + i) * p.num_kb + kb) * 4,
                                                  p.tiles_n * CG * p.num_kb * 4));
                    }
                    if (rank == 0 && !withhold) mbar_arrive_expect_tx(&full[fs], w.narrow ? Cfg::NARROW_TX_AB : Cfg::TX_AB);
                    const uint32_t a_dst = smem_addr(smem + Cfg::OFF_A + s * Cfg::A_BYTES);
                    const uint32_t b_dst = smem_addr(smem + Cfg::OFF_B + s * Cfg::B_BYTES);
                    const int kx = checked_x<Cfg::ELEM_BYTES>(p.status, kb * Cfg::BK, p.num_kb * Cfg::BK);
                    const int my = checked_y(p.status, m0, p.tiles_m * CG * TILE_M);
                    if constexpr (CG == 1) tma_load_2d(a_dst, &tmX, bar, kx, my);
                    else tma_load_2d_pair(a_dst, &tmX, bar, kx, my);
#pragma unroll
                    for (int i = 0; i < Cfg::BOXES; ++i) {
                        if (w.narrow && i >= Cfg::NARROW_BOXES) break;
                        const uint32_t to = b_dst + i * Cfg::BOX_BYTES;
                        if constexpr (Cfg::BACK) {        // W2 [N][F]: 64 of F x 64 of N
                            const int x = checked_x<2>(p.status, w.f0 + ((int)rank * (w.narrow ? Cfg::NARROW_BOXES : Cfg::BOXES) + i) * 64,
                                                       p.tiles_n * Cfg::HN);
                            const int y = checked_y(p.status, kb * Cfg::BK, p.num_kb * Cfg::BK);
                            if constexpr (CG == 1) tma_load_2d(to, &tmW, bar, x, y);
                            else tma_load_2d_pair(to, &tmW, bar, x, y);
                        } else {                          // W [2][F][K]: 64 rows of one half
                            const bool split = CG == 2 && w.narrow;       // g's rows in the leader, u's in its peer
                            const int half = split ? (int)rank : i;
                            const int y = checked_y(p.status, w.f0 + (split ? 0 : 64 * (int)rank), p.tiles_n * Cfg::HN);
                            if constexpr (CG == 1) tma_load_3d(to, &tmW, bar, kx, y, half);
                            else tma_load_3d_pair(to, &tmW, bar, kx, y, half);
                        }
                    }
                    if (++s == STAGES) { s = 0; ph ^= 1u; }
                    if (++fs == Cfg::FULLS) fs = 0;
                }
            }
        }
    } else if (warp == 1 || (Cfg::ISSUERS == 2 && warp == Cfg::SECOND_ISSUER)) {
        // ----------------------------------------------------------- MMA issue
        const int me = warp == 1 ? 0 : 1;
        if (rank == 0 && lane == 0) {
            // descriptors as in gemm_tc_kernel: K-major operands step 32 bytes per MMA, an
            // N-contiguous B MMA_K rows of 128 bytes
            constexpr uint32_t B_LBO = Cfg::BACK ? Cfg::ATOM_BYTES : 16;
            constexpr uint32_t B_STEP = Cfg::BACK ? (Cfg::MMA_K * 128) >> 4 : 2;
            int s = 0, fs = 0, sg = 0;
            uint32_t ph = 0, sgph = 0, acc_it = 0;
            bool ok = true;
            for (int n = unit0; ok && n < p.units; n += unit_step, ++acc_it) {
                const bool narrow = CG == 2 && n >= p.whole;
                const uint32_t idesc = narrow ? p.idesc_narrow : p.idesc;
                const uint32_t b = Cfg::ACC_BUFS == 2 ? (acc_it & 1u) : 0u;
                const uint32_t aph = Cfg::ACC_BUFS == 2 ? ((acc_it >> 1) & 1u) : (acc_it & 1u);
                if (!W.wait<CG == 2>(&tempty[b], aph ^ 1u)) { ok = false; break; }
                tc_fence_after_sync();
                const uint32_t d_tmem = tmem_base + b * Cfg::ACC_COLS + me * BN;
                uint32_t more = 0;                        // the accumulator holds a sum of this tile's
                for (int j = 0; j < kb1 - kb0; ++j) {
                    [[maybe_unused]] const int kb = kb_at(j, kb0, kb1, acc_it);
                    if constexpr (Cfg::GROUPED) {         // a new group of scales
                        if (j == 0 || group_begins<Cfg>(kb, acc_it))
                            if (!W.wait(&sfready[sg], sgph)) { ok = false; break; }
                    }
                    if (Cfg::ISSUERS == 1 || fs % Cfg::ISSUERS == me) {
                        if (!W.wait(&full[fs], ph)) { ok = false; break; }
                        tc_fence_after_sync();
                        const uint64_t ad = smem_desc(smem_addr(smem + Cfg::OFF_A + s * Cfg::A_BYTES), 16, 1024, SWZ_128B);
                        const uint64_t bd = smem_desc(smem_addr(smem + Cfg::OFF_B + s * Cfg::B_BYTES), B_LBO, 1024, SWZ_128B);
                        if constexpr (Cfg::SCALED) {
                            const uint32_t sfa_t = tmem_base + Cfg::SF_COL0 + (Cfg::PACKED ? s : sg * Cfg::SF_GROUP + kb % Cfg::SF_GROUP) * Cfg::SF_SLOT;
                            const uint32_t sfb_t = sfa_t + 4 * Cfg::SF_WORDS;
#pragma unroll
                            for (int k = 0; k < Cfg::BK / Cfg::MMA_K; ++k) {
                                const uint32_t w = (uint32_t)k / 4u, id = (uint32_t)k % 4u;
                                mma_scaled<Cfg::KIND, CG>(d_tmem, ad + 2 * k, bd + 2 * k, idesc | (id << 4) | (id << 29),
                                                          sfa_t + 4 * w, sfb_t + 4 * Cfg::HALVES * w, more | (k != 0));
                            }
                        } else {
#pragma unroll
                            for (int k = 0; k < Cfg::BK / Cfg::MMA_K; ++k)
                                mma_f16<CG>(d_tmem, ad + 2 * k, bd + B_STEP * k, idesc, more | (k != 0));
                        }
                        more = 1;
                        if constexpr (CG == 1) tc_commit<1>(smem_addr(&empty[s]));
                        else tc_commit_pair(smem_addr(&empty[s]), 0x3);
                    }
                    if constexpr (Cfg::GROUPED) {
                        if (j == kb1 - kb0 - 1 || group_begins<Cfg>(kb_at(j + 1, kb0, kb1, acc_it), acc_it)) {
                            tc_commit<1>(smem_addr(&sfempty[sg]));
                            if (++sg == Cfg::SF_RING) { sg = 0; sgph ^= 1u; }
                        }
                    }
                    if (++s == STAGES) s = 0;
                    if (++fs == Cfg::FULLS) { fs = 0; ph ^= 1u; }
                }
                if (!ok) break;
                if constexpr (CG == 1) tc_commit<1>(smem_addr(&tfull[b]));
                else tc_commit_pair(smem_addr(&tfull[b]), 0x3);
            }
            // every MMA this thread issued has finished before teardown
            tc_commit<CG>(smem_addr(drain));
            W.wait(drain, 0, false);
        }
    } else if (Cfg::COPIER && warp >= Cfg::COPY_WARP) {
        // ---------------------------------------------------------- scale copies
        if constexpr (Cfg::PACKED) {
            if (rank == 0 && lane == 0) {
                // (a narrow tile copies what a whole one's second block left in the stage, which no MMA reads)
                int s = 0, fs = 0;
                uint32_t ph = 0;
                bool ok = true;
                for (int n = unit0; ok && n < p.units; n += unit_step) {
                    for (int j = 0; j < kb1 - kb0; ++j) {
                        if (!W.wait(&sffull[s], ph)) { ok = false; break; }
                        tc_fence_after_sync();
                        const uint32_t sfa_t = tmem_base + Cfg::SF_COL0 + s * Cfg::SF_SLOT;
                        copy_scales<Cfg, Cfg::COPIERS>(smem, s, sfa_t, sfa_t + 4 * Cfg::SF_WORDS, warp - Cfg::COPY_WARP);
                        if constexpr (CG == 1) tc_commit<1>(smem_addr(&full[fs]));
                        else tc_commit_pair(smem_addr(&full[fs]), 0x1);
                        if (++s == STAGES) { s = 0; ph ^= 1u; }
                        if (++fs == Cfg::FULLS) fs = 0;
                    }
                }
                // every copy this thread issued has finished before teardown
                if constexpr (CG == 1) tc_commit<1>(smem_addr(cdrain));
                else tc_commit_pair(smem_addr(cdrain), 0x1);
                W.wait(cdrain, 0, false);
            }
        }
        if constexpr (Cfg::GROUPED) {
            // Groups of four k-blocks, numbered over the CTA's units in the order in which the MMAs take them: copying warp c
            // has every COPIERS-th, so that its loads for the next have that long to arrive (the fence between the words
            // and the copies waits for them: with one warp for all groups a k-block took 0.4 us)
            const int sfk = (p.K + rows::BLOCK - 1) / rows::BLOCK;
            const int first = kb0 / Cfg::SF_GROUP, groups = (kb1 - 1) / Cfg::SF_GROUP - first + 1;
            // codes of the rows of a k-block group, 16 of each row: word i of block b is row 32 i + lane.  1.0 stands for
            // rows past the matrix
            struct Group {
                uint4 w[Cfg::SF_BLOCKS][4];
                bool on;
            };
            auto fetch = [&](int64_t t) {                 // the t-th group
                Group r;
                const int turn = (int)(t / groups), i = (int)(t - (int64_t)turn * groups), n = unit0 + turn * unit_step;
                r.on = n < p.units;
                if (!r.on) return r;
                const int g = first + (GB300_SERPENTINE_K && (turn & 1) ? groups - 1 - i : i);
                const GatedUnit w = gated_unit<Cfg>(p, n);
#pragma unroll
                for (int b = 0; b < Cfg::SF_BLOCKS; ++b)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        int64_t row = w.tm * TILE_M + 32 * k + lane;                      // 128 rows of X
                        bool on = row < p.M;
                        if (b > 0) {                                                      // 64 of g's rows, 64 of u's
                            const int f = w.f0 + (b - 1) * 64 + 32 * (k % 2) + lane;
                            row = (int64_t)(k / 2) * p.F + f;
                            on = f < p.F;
                        }
                        r.w[b][k] = make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                        if (on) r.w[b][k] = reinterpret_cast<const uint4 *>((b == 0 ? p.sfx : p.sfw) + row * sfk)[g];
                    }
                return r;
            };
            Group next = fetch(warp - Cfg::COPY_WARP);
            for (int64_t t = warp - Cfg::COPY_WARP; next.on; t += Cfg::COPIERS) {
                const int slot = (int)(t % Cfg::SF_RING);
                const uint32_t ph = (uint32_t)(t / Cfg::SF_RING) & 1u;
                const uint32_t from = smem_addr(smem + Cfg::OFF_SF) + slot * Cfg::SF_GROUP * Cfg::SF_BLOCKS * 512;
                const Group now = next;
                next = fetch(t + Cfg::COPIERS);
                if (!__all_sync(0xffffffffu, W.wait(&sfempty[slot], ph ^ 1u))) break;
#pragma unroll
                for (int b = 0; b < Cfg::SF_BLOCKS; ++b) {
                    const uint4 *q = now.w[b];
                    const uint32_t to = from + 512 * b + 16 * lane;
                    st_shared_v4(to, q[0].x, q[1].x, q[2].x, q[3].x);
                    st_shared_v4(to + Cfg::SF_BLOCKS * 512, q[0].y, q[1].y, q[2].y, q[3].y);
                    st_shared_v4(to + 2 * Cfg::SF_BLOCKS * 512, q[0].z, q[1].z, q[2].z, q[3].z);
                    st_shared_v4(to + 3 * Cfg::SF_BLOCKS * 512, q[0].w, q[1].w, q[2].w, q[3].w);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tc_fence_after_sync();
#pragma unroll
                    for (int k = 0; k < Cfg::SF_GROUP; ++k)
#pragma unroll
                        for (int b = 0; b < Cfg::SF_BLOCKS; ++b)                          // X's, then W's
                            tmem_cp_32x128b_warpx4<CG>(
                                tmem_base + Cfg::SF_COL0 + (slot * Cfg::SF_GROUP + k) * Cfg::SF_SLOT + 4 * b,
                                smem_desc(from + (k * Cfg::SF_BLOCKS + b) * 512, 512, 128, SWZ_NONE));
                    tc_commit<1>(smem_addr(&sfready[slot]));
                }
            }
            if (lane == 0) {                              // every copy this thread issued has finished before teardown
                tc_commit<1>(smem_addr(cdrain));
                W.wait(cdrain, 0, false);
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        const int e = warp - 2;
        const int q = warp & 3;                           // TMEM lane window of this warp
        const int h = e / 4;                              // which WCOLS-wide slice of the tile's columns
        // slices: the CTA that owns the warp's piece (by lane window, with eight slices by column slice too), and its number there
        const int owner = slices == 8 ? 4 * h + q : q * slices / 4;
        const int own = slices == 8 ? 0 : slices == 4 ? h : 2 * (q % 2) + h;
        const uint32_t box = smem_addr(smem + Cfg::OFF_EPI + (Cfg::SLICED ? own : e) * Cfg::EPI_BUF);
        const uint64_t stream_pol = l2_policy_evict_first();
        const int blocks = (p.F + rows::BLOCK - 1) / rows::BLOCK;
        const bool bf16 = p.out16 == GEMM_BF16;
        uint32_t acc_it = 0;
        // hand accumulator b back to the MMA (all 32 lanes have read it)
        auto release = [&](uint32_t b) {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                if constexpr (CG == 1) mbar_arrive(&tempty[b]);
                else mbar_arrive_remote(mapa_shared(smem_addr(&tempty[b]), 0));
            }
        };
        for (int n = unit0; n < p.units; n += unit_step, ++acc_it) {
            const GatedUnit w = gated_unit<Cfg>(p, n);
            const uint32_t b = Cfg::ACC_BUFS == 2 ? (acc_it & 1u) : 0u;
            const uint32_t aph = Cfg::ACC_BUFS == 2 ? ((acc_it >> 1) & 1u) : (acc_it & 1u);
            const int m_warp = (w.tm * CG + (int)rank) * TILE_M + 32 * q;
            const int wchunks = w.narrow ? Cfg::NARROW_WCHUNKS : Cfg::WCHUNKS;
            const int f_warp = w.f0 + h * wchunks * EPI_COLS;
            const int row = m_warp + lane;
            // forward: g's columns of the warp's slice, u's are 64 further on; backward: da's
            const int col = Cfg::BACK ? h * wchunks * EPI_COLS : (w.narrow ? 32 * h : 128 * h);
            const uint32_t taddr = tmem_base + ((uint32_t)(32 * q) << 16) + b * Cfg::ACC_COLS + col;
            // 32 columns' sums, the issuers' added up (of a tile of one k-block only the one whose turn it was has some)
            auto load_sums = [&](uint32_t from, uint32_t (&v)[32]) {
                tmem_ld_32x32b_x32(Cfg::ISSUERS == 2 && kb1 - kb0 == 1 && (acc_it & 1u) ? from + BN : from, v);
                if constexpr (Cfg::ISSUERS == 2) {
                    if (kb1 - kb0 > 1) {
                        uint32_t other[32];
                        tmem_ld_32x32b_x32(from + BN, other);
                        tmem_ld_wait(v);
                        tie_registers(other);
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(other[i]));
                    }
                }
            };
            // chunks with a column of the matrix; none where the warp's rows are all past M
            const int chunks = m_warp < p.M ? max(0, min(wchunks, (p.F - f_warp + EPI_COLS - 1) / EPI_COLS)) : 0;

            // the staging is free again once the last chunk's boxes have been read
            auto begin_boxes = [&]() {
                if (lane == 0) bulk_wait_group_read0();
                __syncwarp();
            };
            auto end_boxes = [&]() {
                fence_proxy_async_smem();
                __syncwarp();
            };

            // Slices: this warp's sums of 32 rows (v: a chunk's 32 columns of one or two accumulators) go to the piece's
            // owner, or are added to the others' there.  False where the piece is another CTA's, or the kernel gives up.
            auto exchange = [&](int c, uint32_t (&v)[Cfg::BACK ? 1 : 2][32]) -> bool {
                if constexpr (!Cfg::SLICED) return true;
                if (c >= chunks) return false;
                const int sets = Cfg::BACK ? 1 : 2, set_bytes = 4096;
                const uint32_t piece = smem_addr(smem + Cfg::OFF_EPI) + (uint32_t)(8 / slices * Cfg::EPI_BUF) +
                                       (uint32_t)(own * (slices - 1) * Cfg::PIECE + c * sets * set_bytes + 16 * lane);
                if (owner != slice) {
                    const uint32_t to = mapa_shared(piece + (uint32_t)(slice - (slice > owner)) * Cfg::PIECE, (uint32_t)owner);
                    const uint32_t bar = mapa_shared(smem_addr(&recv[own]), (uint32_t)owner);
#pragma unroll
                    for (int s = 0; s < sets; ++s)
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            st_async_v4(to + s * set_bytes + 512 * i, v[s][4 * i], v[s][4 * i + 1], v[s][4 * i + 2],
                                        v[s][4 * i + 3], bar);
                    return false;
                }
                if (c == 0) {                             // all chunks of the piece
                    if (lane == 0)
                        mbar_arrive_expect_tx(&recv[own], (uint32_t)((slices - 1) * chunks * sets * set_bytes));
                    if (!__all_sync(0xffffffffu, W.template wait<true>(&recv[own], 0))) return false;
                }
                float sum[Cfg::BACK ? 1 : 2][32] = {};
                for (int k = 0; k < slices; ++k) {
                    const uint32_t at = piece + (uint32_t)(k - (k > slice)) * Cfg::PIECE;
#pragma unroll
                    for (int s = 0; s < sets; ++s)
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            float4 f = make_float4(__uint_as_float(v[s][4 * i]), __uint_as_float(v[s][4 * i + 1]),
                                                   __uint_as_float(v[s][4 * i + 2]), __uint_as_float(v[s][4 * i + 3]));
                            if (k != slice) f = ld_shared_v4f(at + s * set_bytes + 512 * i);
                            sum[s][4 * i] += f.x;
                            sum[s][4 * i + 1] += f.y;
                            sum[s][4 * i + 2] += f.z;
                            sum[s][4 * i + 3] += f.w;
                        }
                }
#pragma unroll
                for (int s = 0; s < sets; ++s)
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[s][i] = __float_as_uint(sum[s][i]);
                return true;
            };

            if constexpr (!Cfg::BACK) {
                const uint32_t box_g = box + 2048, box_u = box_g + 1024;     // behind a's two KiB, a KiB each
                auto finish = [&](int c, const uint32_t (&gr)[32], const uint32_t (&ur)[32]) {
                    if (c >= chunks) return;
                    const int f = f_warp + EPI_COLS * c;
                    float g[32], u[32], a[32];
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float2 g2 = make_float2(__uint_as_float(gr[i]), __uint_as_float(gr[i + 1]));
                        const float2 u2 = make_float2(__uint_as_float(ur[i]), __uint_as_float(ur[i + 1]));
                        float2 s1, s0;
                        rows::sigmoid2(g2, s1, s0);
                        const float2 a2 = rows::mul2(rows::mul2(g2, s1), u2);
                        g[i] = g2.x;
                        g[i + 1] = g2.y;
                        u[i] = u2.x;
                        u[i + 1] = u2.y;
                        a[i] = a2.x;
                        a[i + 1] = a2.y;
                    }
                    begin_boxes();
                    const int64_t block = (int64_t)row * blocks + f / rows::BLOCK;
                    if (p.a_8bit) {
                        const uint32_t code = quantise_chunk(a, box, lane);
                        if (row < p.M) p.sfa[block] = (uint8_t)code;
                    } else {
                        round_chunk(a, bf16, box, lane);
                    }
                    if (p.has_z) {
                        const uint32_t cg = quantise_chunk(g, box_g, lane), cu = quantise_chunk(u, box_u, lane);
                        if (row < p.M) {
                            uint8_t *sf = p.sfck + (block + (int64_t)row * blocks);
                            sf[0] = (uint8_t)cg;
                            sf[blocks] = (uint8_t)cu;
                        }
                    }
                    end_boxes();
                    if (lane == 0) {
                        const int x = checked_x<1>(p.status, f, p.F), y = checked_y(p.status, m_warp, p.M);
                        tma_store_2d_hint(&tmA, box, x, y, stream_pol);
                        if (p.has_z) {
                            tma_store_3d_hint(&tmZ, box_g, x, 0, y, stream_pol);
                            tma_store_3d_hint(&tmZ, box_u, x, 1, y, stream_pol);
                        }
                        bulk_commit_group();
                    }
                };
                if (!__all_sync(0xffffffffu, W.wait(&tfull[b], aph))) break;
                tc_fence_after_sync();
                if constexpr (Cfg::ACC_BUFS == 1 && Cfg::WCHUNKS > 1) {
                    // the whole slice to registers first, so that the MMA can start the next tile
                    uint32_t g[Cfg::WCHUNKS][32], u[Cfg::WCHUNKS][32];
#pragma unroll
                    for (int c = 0; c < Cfg::WCHUNKS; ++c) {
                        if (c >= wchunks) break;
                        tmem_ld_32x32b_x32(taddr + EPI_COLS * c, g[c]);
                        tmem_ld_32x32b_x32(taddr + 64 + EPI_COLS * c, u[c]);
                    }
                    tmem_ld_wait_all();
#pragma unroll
                    for (int c = 0; c < Cfg::WCHUNKS; ++c) {
                        tie_registers(g[c]);
                        tie_registers(u[c]);
                    }
                    release(b);
#pragma unroll
                    for (int c = 0; c < Cfg::WCHUNKS; ++c) finish(c, g[c], u[c]);
                } else {
#pragma unroll 1
                    for (int c = 0; c < wchunks; ++c) {
                        uint32_t v[2][32];
                        load_sums(taddr + EPI_COLS * c, v[0]);
                        load_sums(taddr + 64 + EPI_COLS * c, v[1]);
                        tmem_ld_wait(v[0]);
                        tie_registers(v[1]);
                        if (c == wchunks - 1) release(b);
                        if (exchange(c, v)) finish(c, v[0], v[1]);
                    }
                }
            } else {
                // codes and scales of a chunk's g and u; zeros past the matrix
                struct Kept {
                    uint4 g[2], u[2];
                    uint32_t sg, su;
                };
                auto fetch = [&](int c) {
                    Kept k{};
                    const int f = f_warp + EPI_COLS * c;
                    if (c < chunks && row < p.M) {
                        const uint8_t *ck = p.ck + (int64_t)row * 2 * p.F + f;
                        const uint8_t *sf = p.sfck_in + (int64_t)row * 2 * blocks + f / rows::BLOCK;
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            if (f + 16 * i < p.F) {
                                k.g[i] = *reinterpret_cast<const uint4 *>(ck + 16 * i);
                                k.u[i] = *reinterpret_cast<const uint4 *>(ck + p.F + 16 * i);
                            }
                        k.sg = sf[0];
                        k.su = sf[blocks];
                    }
                    return k;
                };
                Kept next = fetch(0);
                if (!__all_sync(0xffffffffu, W.wait(&tfull[b], aph))) break;
                tc_fence_after_sync();
#pragma unroll 1
                for (int c = 0; c < wchunks; ++c) {
                    const Kept k = next;
                    if (c + 1 < wchunks) next = fetch(c + 1);
                    uint32_t v[1][32];
                    load_sums(taddr + EPI_COLS * c, v[0]);
                    tmem_ld_wait(v[0]);
                    if (c == wchunks - 1) release(b);
                    if (c >= chunks || !exchange(c, v)) continue;
                    begin_boxes();
                    const float sg = rows::scale_value(k.sg), su = rows::scale_value(k.su);
#pragma unroll
                    for (int o = 0; o < 4; ++o) {         // eight columns at a time
                        const uint4 gq = k.g[o / 2], uq = k.u[o / 2];
                        float g[8], u[8], dg[8], du[8], a[8];
                        rows::decode(o % 2 ? make_uint2(gq.z, gq.w) : make_uint2(gq.x, gq.y), sg, g);
                        rows::decode(o % 2 ? make_uint2(uq.z, uq.w) : make_uint2(uq.x, uq.y), su, u);
#pragma unroll
                        for (int i = 0; i < 8; i += 2) {
                            using namespace rows;
                            const float2 da = make_float2(__uint_as_float(v[0][8 * o + i]), __uint_as_float(v[0][8 * o + i + 1]));
                            const float2 g2 = make_float2(g[i], g[i + 1]), u2 = make_float2(u[i], u[i + 1]);
                            float2 s1, s0;
                            sigmoid2(g2, s1, s0);
                            const float2 gs = mul2(g2, s1), a2 = mul2(gs, u2), du2 = mul2(da, gs);
                            const float2 dg2 = mul2(mul2(da, u2), mul2(s1, fma2(g2, s0, both(1.f))));
                            a[i] = a2.x;
                            a[i + 1] = a2.y;
                            dg[i] = dg2.x;
                            dg[i + 1] = dg2.y;
                            du[i] = du2.x;
                            du[i + 1] = du2.y;
                        }
                        auto put = [&](uint32_t to, const float (&v)[8]) {
                            const uint4 w = bf16 ? rows::pack8(static_cast<const __nv_bfloat16 *>(nullptr), v)
                                                 : rows::pack8(static_cast<const __half *>(nullptr), v);
                            st_shared_v4(to + swz_off<64>(lane, o), w.x, w.y, w.z, w.w);
                        };
                        put(box, dg);
                        put(box + 2048, du);
                        if (p.has_a) put(box + 4096, a);
                    }
                    end_boxes();
                    if (lane == 0) {
                        const int x = checked_x<2>(p.status, f_warp + EPI_COLS * c, p.F), y = checked_y(p.status, m_warp, p.M);
                        tma_store_3d_hint(&tmZ, box, x, 0, y, stream_pol);
                        tma_store_3d_hint(&tmZ, box + 2048, x, 1, y, stream_pol);
                        if (p.has_a) tma_store_2d_hint(&tmA, box + 4096, x, y, stream_pol);
                        bulk_commit_group();
                    }
                }
            }
        }
        if (lane == 0) bulk_wait_group0();
    }

    // ----------------------------------------------------------------- teardown
    __syncwarp();
    if (*abort_flag) {
        // give copies that were already in flight time to land before the
        // shared memory they target is released
        for (int i = 0; i < 64; ++i) __nanosleep(1000);
    }
    tc_fence_before_sync();
    // (slices: no CTA leaves while another may still send it sums)
    if constexpr (CG == 2 || Cfg::SLICED) cluster_sync(); else __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc<CG>(tmem_base, 512);
    }
}

// What the host does with an instance
template <class Cfg>
struct GatedInstance {
    static GatedShape shape() { return {Cfg::HN, Cfg::STAGES, Cfg::SMEM_BYTES, Cfg::BK}; }
    // the most clusters of `slices` CTAs (pairs: of two) that run at once
    static cudaError_t prepare(int slices, int *clusters) {
        const void *f = reinterpret_cast<const void *>(&gated_kernel<Cfg>);
        cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t lc = config(2 * 1024, nullptr);
        cudaLaunchAttribute attr = cluster(slices);
        lc.attrs = &attr;
        lc.numAttrs = 1;
        return cudaOccupancyMaxActiveClusters(clusters, f, &lc);
    }
    static cudaError_t launch(int grid, const CUtensorMap *maps, const GatedParams &p, cudaStream_t stream) {
        cudaLaunchConfig_t lc = config(grid, stream);
        cudaLaunchAttribute attr[2] = {cluster(p.slices), {}};
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        lc.attrs = attr;
        lc.numAttrs = 2;
        return cudaLaunchKernelEx(&lc, gated_kernel<Cfg>, maps[0], maps[1], maps[4], maps[5], maps[2], maps[3], p);
    }

private:
    static cudaLaunchConfig_t config(int grid, cudaStream_t stream) {
        cudaLaunchConfig_t lc = {};
        lc.gridDim = dim3((unsigned)grid);
        lc.blockDim = dim3(Cfg::THREADS);
        lc.dynamicSmemBytes = Cfg::SMEM_BYTES;
        lc.stream = stream;
        return lc;
    }
    static cudaLaunchAttribute cluster(int slices) {
        cudaLaunchAttribute a = {};
        a.id = cudaLaunchAttributeClusterDimension;
        a.val.clusterDim.x = Cfg::SLICED ? (unsigned)slices : (unsigned)Cfg::CG;
        a.val.clusterDim.y = a.val.clusterDim.z = 1;
        return a;
    }
};

}  // namespace gb300
