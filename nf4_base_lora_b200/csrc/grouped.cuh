// The fused NF4-LoRA products over ragged row groups, on tcgen05:
//
//   forward        Y_i  = X_i W_e^T + T_i B_e^T                  rows i of group e
//   input gradient dX_i = dY_i W_e  + gain keep_i .* (V_i A_e)   (keep: adapter dropout)
//
// The weight is the MMA's M side and the rows of the group (tokens) its N side:
// D^T[weight column, token].  A cluster of two CTAs computes 256 weight columns
// by up to T tokens of one group with MMAs over the pair (cta_group::2, M = 256,
// N = 32 .. 256): each CTA decodes 128 of the 256 weight columns and holds half
// of the tokens, both in its own shared memory, and the accumulators of its 128
// weight columns in its own tensor memory.  So a decoded weight serves up to 512
// tokens (two accumulators of 256 columns), more than one CTA's tensor memory
// would allow in the other orientation, and N follows the group's real size in
// steps of 32: a ragged tail costs little and one kernel serves groups of one
// token and of thousands.
//
// The groups' bounds are device data, so the grid covers the most token tiles
// any split of M rows into E groups can need; each warp finds its tile by a scan
// of the offsets, and a pair beyond the last tile leaves.  A tile never crosses
// a group: rows of the next group that its copies bring in are accumulator
// columns that are not stored, or beyond N altogether.
//
// Weights and factors are three-dimensional tensor maps (inner, row, expert):
// rows beyond an expert's own read as zeros and never as the next expert's, so
// a NaN or an infinity in one expert's adapter cannot reach another's result.
//
// Warp roles, in each CTA: warp 0 copies (TMA, one lane); warp 1 owns tensor
// memory, and in the leading CTA its first lane issues the MMAs; teams of four
// warps decode k-steps in turn (one (weight row, block) unit per thread, register
// codebook) and then run the epilogue.  The rank-r term enters the same
// accumulator as extension k-steps over [hi | lo] of the 16-bit pair of T or V.
//
// Dropout (input gradient): the extension steps come first, the epilogue warps
// read the accumulators back, keep and scale them in fp32 and store them to
// tensor memory, and the base product then accumulates on top.  The mask costs
// no memory traffic and the rank-r term no second output pass.
#pragma once

#include <cstdint>

#include "gemm.cuh"
#include "philox.cuh"

namespace nf4lora {

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int32_t x,
                                            int32_t y, int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 lanes x 8 columns of fp32.
__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}

// ------------------------------------------------------------------ groups
struct GroupTile {
    int e;        // expert
    int row0;     // first row of the tile
    int row_end;  // end of the group's rows
};

// Bounds of group e, clamped into 0 <= begin <= end <= M, so that offsets that
// break the contract can never lead an access out of the arrays.
__device__ __forceinline__ void group_bounds(const int32_t* offsets, int e, int M, int& begin, int& end) {
    begin = min(max(__ldcg(offsets + e), 0), M);
    end = min(max(__ldcg(offsets + e + 1), begin), M);
}

// Tile t of all groups' tiles of `tile_rows` rows, in group order; the whole
// warp calls it.  False beyond the last tile.
__device__ __forceinline__ bool find_tile(const int32_t* offsets, int E, int M, int tile_rows, int t, int lane,
                                          GroupTile& g) {
    if (offsets == nullptr) {
        g.e = 0;
        g.row0 = t * tile_rows;
        g.row_end = M;
        return g.row0 < M;
    }
    int before = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
        const int e = e0 + lane;
        int begin = 0, end = 0;
        if (e < E) group_bounds(offsets, e, M, begin, end);
        const int n = (end - begin + tile_rows - 1) / tile_rows;
        int incl = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
            if (lane >= d) incl += v;
        }
        const unsigned hit = __ballot_sync(0xFFFFFFFFu, before + incl > t);
        if (hit != 0) {
            const int src = __ffs(hit) - 1;
            g.e = e0 + src;
            const int excl = __shfl_sync(0xFFFFFFFFu, incl - n, src);
            g.row0 = __shfl_sync(0xFFFFFFFFu, begin, src) + (t - before - excl) * tile_rows;
            g.row_end = __shfl_sync(0xFFFFFFFFu, end, src);
            return true;
        }
        before += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    return false;
}

// ------------------------------------------------------------------ CTA pairs
__device__ __forceinline__ void mma2_bf16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrive once on `bar` of both CTAs of the pair when every MMA issued so far by
// this thread has completed.
__device__ __forceinline__ void mma2_commit(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

// Arrive on a barrier of either CTA of the pair (a shared::cluster address).
// The default form, at CTA scope: what it publishes are operand tiles that only
// MMAs read, ordered for them by the proxy fence before it, and accumulators,
// ordered by the tcgen05 fences; a cluster-scope release would add a memory
// barrier to every arrival.
__device__ __forceinline__ void mbar_arrive_pair(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Allocation and release of the same columns in both CTAs; a warp of each calls it.
__device__ __forceinline__ void tmem2_alloc(uint32_t* dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem2_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// ------------------------------------------------------------------ fused product
struct GroupGemmArgs {
    const int32_t* offsets;  // [E + 1], or NULL
    int E;
    int M;
    int cols;                // forward: N; input gradient: K
    int k_main;              // 64-wide steps of the contraction
    int k_ext;               // extension steps: 2 r64 / 64
    int cols_fastest;        // 1: the pairs along grid.x walk the column tiles, else the row tiles
    // encoded weight: rows and blocks of one expert
    const int8_t* qscale;
    const float* scale2;
    const float* scale_mean;
    const float* absmax;
    int w_rows;
    int w_blocks_per_row;
    uint16_t* out;           // [M, cols]
    DropArgs drop;           // input gradient with dropout only
};

// T tokens per tile.  512: one CTA per SM, four teams; 128 and 64: two CTAs per
// SM of two teams each, whose starts and ends overlap.
template <bool DX, int T>
struct GroupGemmConfig {
    static constexpr int kBM = 128;                    // weight columns of one CTA
    static constexpr int kSubs = T > 256 ? 2 : 1;      // accumulators
    static constexpr int kSubT = T / kSubs;            // tokens of one, half of them per CTA
    static constexpr int kTeams = T > 128 ? 4 : 2;
    static constexpr int kDS = T == 128 ? 2 : 4;       // decoded tiles of 16 KB
    static constexpr int kLS = 4;                      // load slots: codes and tokens
    static constexpr int kSub = kSubT / 2 * 128;       // a CTA's tokens of one accumulator, 64 deep
    static constexpr int kTokBytes = kSubs * kSub;
    static constexpr int kCBytes = kBM * 32;           // packed codes of a step
    static constexpr int kWBytes = kBM * 128;          // decoded tile
    static constexpr int kLoadSlot = kTokBytes + kCBytes;
    static constexpr int kSmem = kLS * kLoadSlot + kDS * kWBytes + 1024;
    static constexpr int kTeamThreads = kBM;           // one (row, block) unit each
    static constexpr int kTeamWarps = kTeamThreads / 32;
    static constexpr int kWorkWarps = kTeamWarps * kTeams;
    static constexpr int kThreads = 64 + 32 * kWorkWarps;
    static constexpr int kMinBlocks = T > 128 ? 1 : 2;
    static constexpr int kTmemCols = T < 32 ? 32 : T;
    static constexpr uint32_t kIdesc = make_idesc_bf16(2 * kBM, 0, DX ? 1 : 0, 0);  // without N
    static_assert(kLS <= 2 * kDS, "the copies' waits on a decode slot could not tell its phases apart");
    static_assert(kLS % kTeams == 0 && kDS % kTeams == 0, "a ring slot is one team's");
    static_assert(kLoadSlot % 1024 == 0 && kSmem * kMinBlocks <= 226 * 1024, "shared memory");
};

// map_t: X [M, K] or dY [M, N], box {64, kSubT / 2}.  map_w: codes (K / 2, N,
// E), box {32, 128, 1} (forward) or {64, 64, 1}.  map_te: T2 or V2 [M, 2 r64],
// box {64, kSubT / 2}.  map_we: B (r, N, E), box {64, 128, 1} (forward) or A (K,
// r, E), box {64, 64, 1}.  Cluster of two along grid.x.
template <bool DX, int T, bool DROP>
__global__ void __launch_bounds__(GroupGemmConfig<DX, T>::kThreads, GroupGemmConfig<DX, T>::kMinBlocks)
    k_group_gemm(const __grid_constant__ CUtensorMap map_t, const __grid_constant__ CUtensorMap map_w,
                 const __grid_constant__ CUtensorMap map_te, const __grid_constant__ CUtensorMap map_we,
                 const GroupGemmArgs args) {
    using C = GroupGemmConfig<DX, T>;
    static_assert(DX || !DROP, "only the input gradient masks its accumulator");
    constexpr int LS = C::kLS, DS = C::kDS;
    constexpr int kWork = C::kWorkWarps * 32;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    // bar_ready and bar_masked count both CTAs' arrivals, in the leading CTA
    // (rank 0); the rest are each CTA's own, and the MMAs' completions arrive in
    // both
    __shared__ uint64_t bar_full[LS], bar_empty[LS], bar_ready[DS], bar_dempty[DS], bar_accum, bar_ext,
        bar_masked;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // the offsets, the activations and the encoded weight were complete before
    // the kernel this one depends on released it (that kernel waited for all
    // earlier ones first); T2 / V2 is that kernel's and is waited for below
    GroupTile g;
    const int pair = blockIdx.x >> 1;
    const int ct = args.cols_fastest ? pair : blockIdx.y;
    const int rt = args.cols_fastest ? blockIdx.y : pair;
    if (!find_tile(args.offsets, args.E, args.M, T, rt, lane, g)) {
        // every CTA waits, so this grid's completion implies the earlier kernels'
        grid_dependency_wait();
        return;
    }
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* base = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    auto t_buf = [&](int it) { return base + (it % LS) * C::kLoadSlot; };
    auto codes_buf = [&](int it) { return base + (it % LS) * C::kLoadSlot + C::kTokBytes; };
    auto w_buf = [&](int it) { return base + LS * C::kLoadSlot + (it % DS) * C::kWBytes; };
    const int h0 = (2 * ct + rank) * C::kBM;  // weight columns of this CTA
    const int tokens = min(T, g.row_end - g.row0);
    const int nsub = C::kSubs == 2 && tokens > C::kSubT ? 2 : 1;
    // N of accumulator s, and the first of the rows that this CTA brings for it
    auto sub_n = [&](int s) { return (min(C::kSubT, tokens - s * C::kSubT) + 31) & ~31; };
    auto sub_row = [&](int s) { return g.row0 + s * C::kSubT + rank * (sub_n(s) >> 1); };
    const int n_main = args.k_main, n_ext = args.k_ext, n_iter = n_main + n_ext;
    // iteration it: the extension steps come last, or first with dropout
    auto is_main = [&](int it) { return DROP ? it >= n_ext : it < n_main; };
    const int main0 = DROP ? n_ext : 0, ext0 = DROP ? 0 : n_main;

    if (threadIdx.x == 0) {
        for (int i = 0; i < LS; ++i) {
            mbar_init(&bar_full[i], 1);
            mbar_init(&bar_empty[i], 1);
        }
        for (int i = 0; i < DS; ++i) {
            mbar_init(&bar_ready[i], 2 * C::kTeamWarps);
            mbar_init(&bar_dempty[i], 1);
        }
        mbar_init(&bar_accum, 1);
        mbar_init(&bar_ext, 1);
        mbar_init(&bar_masked, 2 * C::kWorkWarps);
        s_abort = 0;
        fence_barrier_init();
    }
    // both CTAs' barriers are initialised once the cluster barrier is passed;
    // thread 0, the producer, touches only its own and goes straight on
    cluster_arrive_release();
    if (threadIdx.x != 0) cluster_wait_acquire();
    volatile int* abort_flag = &s_abort;
    // the leading CTA's copy of a barrier (shared::cluster address)
    auto lead = [&](uint64_t* bar) { return cluster_map(smem_u32(bar), 0); };

    if (warp == 0) {
        // ------------------------------------------------------------ copies
        if (lane == 0) {
            tma_prefetch_desc(&map_t);
            tma_prefetch_desc(&map_w);
            tma_prefetch_desc(&map_te);
            tma_prefetch_desc(&map_we);
            int issued = 0;
            for (int it = 0; it < n_iter; ++it) {
                if (it >= LS && !mbar_wait(&bar_empty[it % LS], ((it / LS) & 1u) ^ 1u, abort_flag)) break;
                if (*abort_flag) break;
                uint64_t* bar = &bar_full[it % LS];
                if (is_main(it)) {
                    const int kb = it - main0;
                    mbar_arrive_expect_tx(bar, nsub * C::kSub + C::kCBytes);
                    for (int ms = 0; ms < nsub; ++ms)
                        tma_load_2d(t_buf(it) + ms * C::kSub, &map_t, bar, kb * 64, sub_row(ms));
                    if constexpr (DX) tma_load_3d(codes_buf(it), &map_w, bar, h0 / 2, kb * 64, g.e);
                    else tma_load_3d(codes_buf(it), &map_w, bar, kb * 32, h0, g.e);
                } else {
                    const int j = it - ext0;
                    // the factor's tile lands in a decode slot
                    if (it >= DS && !mbar_wait(&bar_dempty[it % DS], ((it / DS) & 1u) ^ 1u, abort_flag)) break;
                    if (j == 0) grid_dependency_wait();
                    const int jb = j % (n_ext / 2);  // [hi | lo] against the factor twice
                    mbar_arrive_expect_tx(bar, nsub * C::kSub + C::kWBytes);
                    for (int ms = 0; ms < nsub; ++ms)
                        tma_load_2d(t_buf(it) + ms * C::kSub, &map_te, bar, j * 64, sub_row(ms));
                    if constexpr (DX) {
#pragma unroll
                        for (int c = 0; c < C::kBM / 64; ++c)
                            tma_load_3d(w_buf(it) + c * 8192, &map_we, bar, h0 + c * 64, jb * 64, g.e);
                    } else {
                        tma_load_3d(w_buf(it), &map_we, bar, jb * 64, h0, g.e);
                    }
                }
                ++issued;
            }
            if (*abort_flag) {
                // let the copies already issued land before the CTA exits
                for (int it = issued > LS ? issued - LS : 0; it < issued; ++it)
                    mbar_drain(&bar_full[it % LS], (it / LS) & 1u);
            }
            cluster_wait_acquire();  // the first phase, which every other thread passed at the start
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ tensor memory, MMAs
        tmem2_alloc(&s_tmem, C::kTmemCols);
        tc_fence_before();
        asm volatile("bar.arrive 2, %0;" ::"r"(32 + kWork) : "memory");
        __syncwarp();
        tc_fence_after();
        const uint32_t tmem_d = s_tmem;
        if (lane == 0 && rank == 0) {
            uint32_t idesc[2];
            for (int ms = 0; ms < 2; ++ms) idesc[ms] = C::kIdesc | (static_cast<uint32_t>(max(32, sub_n(ms)) >> 3) << 17);
            for (int it = 0; it < n_iter; ++it) {
                // both CTAs' operands are in place: the one wait of a step
                if (!mbar_wait(&bar_ready[it % DS], (it / DS) & 1u, abort_flag)) break;
                if (DROP && it == main0 && !mbar_wait(&bar_masked, 0, abort_flag)) break;
                tc_fence_after();
                const uint32_t w_base = smem_u32(w_buf(it)), t_base = smem_u32(t_buf(it));
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const uint64_t wdesc = tile_desc(w_base, DX, kk);
                    for (int ms = 0; ms < nsub; ++ms)
                        mma2_bf16_ss(tmem_d + ms * C::kSubT, wdesc, tile_desc(t_base + ms * C::kSub, false, kk),
                                     idesc[ms], it * 4 + kk > 0 ? 1u : 0u);
                }
                mma2_commit(&bar_empty[it % LS]);
                mma2_commit(&bar_dempty[it % DS]);
                if (DROP && it == n_ext - 1) mma2_commit(&bar_ext);
            }
            mma2_commit(&bar_accum);
        }
        __syncwarp();
    } else {
        const int ew = warp - 2;
        const int q = warp & 3;  // tensor memory lane quadrant of this warp
        constexpr int kShare = C::kSubT / (C::kWorkWarps / 4);  // tokens of an accumulator per warp
        static_assert(kShare % 32 == 0, "whole loads of 32 tokens");
        const int tbeg = (ew / 4) * kShare;
        uint32_t tmem_d = 0;
        // keep and scale V A, this warp's part of both accumulators
        auto mask_accumulators = [&]() {
            asm volatile("bar.sync 2, %0;" ::"r"(32 + kWork) : "memory");
            tc_fence_after();
            tmem_d = s_tmem;
            KeepGen gen;
            grid_dependency_wait();  // the generator's state may be as young as V
            gen.init(args.drop);
            if (mbar_wait(&bar_ext, 0, abort_flag)) {
                tc_fence_after();
                const int col = h0 + q * 32 + lane;
                for (int ms = 0; ms < nsub; ++ms) {
#pragma unroll 1
                    for (int tt = tbeg; tt < tbeg + kShare && ms * C::kSubT + tt < tokens; tt += 32) {
                        const uint32_t at = tmem_d + (static_cast<uint32_t>(q * 32) << 16) + ms * C::kSubT + tt;
                        uint32_t v[32];
                        tmem_ld_32x32b_x32(at, v);
                        tmem_ld_wait();
                        const int64_t row0 = g.row0 + ms * C::kSubT + tt;
#pragma unroll
                        for (int o = 0; o < 4; ++o) {
                            // the eight lanes of a generator group draw it for eight
                            // tokens, one each, and exchange the decisions
                            uint32_t f[4];
                            gen.flags(static_cast<uint64_t>((row0 + 8 * o + (lane & 7)) * args.cols + (col & ~7)) >> 3, f);
                            uint32_t bits = 0;
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                bits |= ((f[i] >> 15) & 1u) << (2 * i) | (f[i] >> 31) << (2 * i + 1);
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const uint32_t b = __shfl_sync(0xFFFFFFFFu, bits, (lane & 24) | i);
                                uint32_t& x = v[8 * o + i];
                                x = (b >> (lane & 7)) & 1u ? __float_as_uint(__uint_as_float(x) * args.drop.gain) : 0u;
                            }
                        }
                        tmem_st_32x32b_x32(at, v);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_pair(lead(&bar_masked));
        };
        // ------------------------------------------------------------ decoders
        {
            const int team = ew / C::kTeamWarps;
            const int dt = threadIdx.x - 64 - team * C::kTeamThreads;
            const bool fp32_scales = args.absmax != nullptr;  // no double quantisation
            const float mu = fp32_scales ? 0.0f : __ldg(args.scale_mean);
            // This thread's unit of a step.  Forward: weight row h0 + dt, block
            // kb.  Input gradient: weight row 64 kb + n_local, block cblk of this
            // CTA's half, dealt so that the eight threads of a quarter warp store
            // to distinct bank groups and read codes at most two to one.
            constexpr int kCB = C::kBM / 64;
            static_assert(kCB == 2, "unit mapping");
            int n_local = dt, cblk = 0;
            if constexpr (DX) {
                const int qw = dt >> 3, i = dt & 7;
                n_local = 8 * (qw >> 1) + i;
                cblk = ((i >> 1) + qw) & 1;
            }
            const int dst_off = DX ? cblk * 8192 + n_local * 128 : dt * 128;
            const int swz = DX ? n_local & 7 : dt & 7;
            const int code_off = DX ? (n_local * kCB + cblk) * 32 : dt * 32;
            const int64_t scale_row0 = static_cast<int64_t>(g.e) * args.w_rows;
            // block scales are fetched kPf of this team's steps ahead
            constexpr int kPf = 4;
            int8_t q_pf[kPf];
            float a2_pf[kPf];
            bool ok_pf[kPf];
            auto fetch = [&](int kb, int slot) {
                const int wrow = DX ? kb * 64 + n_local : h0 + dt;
                const int wblk = DX ? h0 / 64 + cblk : kb;
                ok_pf[slot] = kb >= 0 && kb < n_main && wrow < args.w_rows && wblk < args.w_blocks_per_row;
                if (ok_pf[slot]) {
                    const int64_t b = (scale_row0 + wrow) * args.w_blocks_per_row + wblk;
                    if (fp32_scales) {
                        q_pf[slot] = 0;
                        a2_pf[slot] = __ldg(args.absmax + b);
                    } else {
                        q_pf[slot] = __ldg(args.qscale + b);
                        a2_pf[slot] = __ldg(args.scale2 + (b >> 8));
                    }
                }
            };
#pragma unroll
            for (int u = 0; u < kPf; ++u) fetch(team + u * C::kTeams - main0, u);
            bool stop = false, masked = !DROP;
            // a ring slot is always the same team's, so its waits see every phase
            for (int it0 = team; it0 < n_iter && !stop; it0 += kPf * C::kTeams) {
#pragma unroll
                for (int u = 0; u < kPf; ++u) {
                    const int it = it0 + u * C::kTeams;
                    if (it >= n_iter) break;
                    const bool valid = ok_pf[u];
                    const float sc =
                        valid ? (fp32_scales ? a2_pf[u] : nf4_block_scale(q_pf[u], a2_pf[u], mu)) : 0.0f;
                    fetch(it - main0 + kPf * C::kTeams, u);
                    if (DROP && !masked && it >= n_ext) {
                        masked = true;
                        mask_accumulators();
                    }
                    if (!mbar_wait(&bar_full[it % LS], (it / LS) & 1u, abort_flag)) {
                        stop = true;
                        break;
                    }
                    if (is_main(it)) {
                        if (it >= DS && !mbar_wait(&bar_dempty[it % DS], ((it / DS) & 1u) ^ 1u, abort_flag)) {
                            stop = true;
                            break;
                        }
                        uint8_t* dst = w_buf(it) + dst_off;
                        if (!valid) zero_row(dst);
                        else decode_unit_reg(codes_buf(it) + code_off, sc, dst, swz);
                    }
                    // also on an extension step, whose operands the copies brought
                    // whole: the arrival passes on that they have landed
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_pair(lead(&bar_ready[it % DS]));
                }
            }
            if (DROP && !masked) mask_accumulators();
        }
        // ------------------------------------------------------------ epilogue
        if constexpr (!DROP) {
            asm volatile("bar.sync 2, %0;" ::"r"(32 + kWork) : "memory");
            tc_fence_after();
            tmem_d = s_tmem;
        }
        const bool ok = mbar_wait(&bar_accum, 0, abort_flag);
        tc_fence_after();
        if (ok && !*abort_flag) {
            // lane: weight column; a pair of lanes swaps halves of two tokens'
            // values, so that a store writes two tokens' 64-byte runs
            const int col = h0 + q * 32 + (lane & 30), odd = lane & 1;
            for (int ms = 0; ms < nsub; ++ms) {
#pragma unroll 1
                for (int tt = tbeg; tt < tbeg + kShare && ms * C::kSubT + tt < tokens; tt += 32) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(tmem_d + (static_cast<uint32_t>(q * 32) << 16) + ms * C::kSubT + tt, v);
                    tmem_ld_wait();
                    const int row = g.row0 + ms * C::kSubT + tt + odd;
                    uint16_t* dst = args.out + static_cast<int64_t>(row) * args.cols + col;
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const float give = __uint_as_float(odd ? v[j] : v[j + 1]);
                        const float got = __shfl_xor_sync(0xFFFFFFFFu, give, 1);
                        const uint32_t two = odd ? pack_bf16x2(got, __uint_as_float(v[j + 1]))
                                                 : pack_bf16x2(__uint_as_float(v[j]), got);
                        // cols is a multiple of 8
                        if (row + j < g.row_end && col < args.cols)
                            *reinterpret_cast<uint32_t*>(dst + static_cast<int64_t>(j) * args.cols) = two;
                    }
                }
            }
        }
    }
    // neither CTA frees its tensor memory or leaves while the other may still
    // use it, read its operands or arrive on its barriers
    tc_fence_before();
    cluster_arrive_release();
    cluster_wait_acquire();
    if (warp == 1) {
        tc_fence_after();
        tmem2_dealloc(s_tmem, C::kTmemCols);
    }
}

}  // namespace nf4lora
