// The fused NF4-LoRA products over ragged row groups, on tcgen05:
//
//   forward        Y_i  = X_i W_e^T + T_i B_e^T                  rows i of group e
//   input gradient dX_i = dY_i W_e  + gain keep_i .* (V_i A_e)   (keep: adapter dropout)
//
// One CTA computes a (128 MSUB) x 256 tile of one group: MSUB accumulators of
// 128 x 256 that share every decoded weight tile.  The groups' bounds are
// device data, so the grid covers the most row tiles any split of M rows into E
// groups can need; each warp finds its tile by a scan of the offsets, and a
// CTA beyond the last tile leaves.  A tile never crosses a group: rows of the
// next group that its copies bring in stay in accumulator rows that are not
// stored.  In a tile with at most 128 rows the second accumulator is skipped.
//
// Weights and factors are three-dimensional tensor maps (inner, row, expert):
// rows beyond an expert's own read as zeros and never as the next expert's, so
// a NaN or an infinity in one expert's adapter cannot reach another's result.
//
// Warp roles: warp 0 copies (TMA, one lane), warp 1 owns tensor memory and
// issues the MMAs, two teams of eight warps decode alternate k-steps (one
// (weight row, block) unit per thread, register codebook) and then run the
// epilogue.  The rank-r term enters the same accumulator as extension k-steps
// over [hi | lo] of the 16-bit pair of T or V.
//
// Dropout (input gradient): the extension steps come first, the epilogue warps
// read the accumulators back, keep and scale them in fp32 and store them to
// tensor memory, and the base product then accumulates on top.  The mask costs
// no memory traffic and the rank-r term no second output pass; a 256 x 256
// tile's masking is about 2 us beside 80 us of base product at 4096 rows of
// weight.
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

// ------------------------------------------------------------------ fused product
struct GroupGemmArgs {
    const int32_t* offsets;  // [E + 1], or NULL
    int E;
    int M;
    int cols;                // forward: N; input gradient: K
    int k_main;              // 64-wide steps of the contraction
    int k_ext;               // extension steps: 2 r64 / 64
    int cols_fastest;        // as GemmArgs
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

template <bool DX, int MSUB>
struct GroupGemmConfig {
    static constexpr int kBM = 128, kBN = 256;
    static constexpr int kRows = kBM * MSUB;
    static constexpr int kTeams = 2;
    // 256-row tiles: 4 load slots of 40 KB and 2 decoded tiles of 32 KB;
    // 128-row tiles: 4 load slots of 24 KB and 4 decoded tiles
    static constexpr int kLS = 4;
    static constexpr int kDS = MSUB == 2 ? 2 : 4;
    static constexpr int kSub = kBM * 128;             // one 128 x 64 bf16 operand tile
    static constexpr int kABytes = MSUB * kSub;
    static constexpr int kCBytes = kBN * 32;           // packed codes of a step
    static constexpr int kBBytes = kBN * 128;
    static constexpr int kLoadSlot = kABytes + kCBytes;
    static constexpr int kSmem = kLS * kLoadSlot + kDS * kBBytes + 1024;
    static constexpr int kTeamThreads = kBN;           // one (row, block) unit each
    static constexpr int kTeamWarps = kTeamThreads / 32;
    static constexpr int kWorkWarps = kTeamWarps * kTeams;
    static constexpr int kThreads = 64 + 32 * kWorkWarps;
    static constexpr int kTmemCols = kBN * MSUB;
    static constexpr uint32_t kIdesc = make_idesc_bf16(kBM, kBN, 0, DX ? 1 : 0);
    static_assert(kLS <= 2 * kDS, "load ring too deep for the decode ring");
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

// map_a: X [M, K] or dY [M, N], box {64, 128}.  map_w: codes (K / 2, N, E),
// box {32, 256, 1} (forward) or {128, 64, 1}.  map_ae: T2 or V2 [M, 2 r64], box
// {64, 128}.  map_be: B (r, N, E), box {64, 256, 1} (forward) or A (K, r, E),
// box {64, 64, 1}.
template <bool DX, int MSUB, bool DROP>
__global__ void __launch_bounds__(GroupGemmConfig<DX, MSUB>::kThreads, 1)
    k_group_gemm(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w,
                 const __grid_constant__ CUtensorMap map_ae, const __grid_constant__ CUtensorMap map_be,
                 const GroupGemmArgs args) {
    using C = GroupGemmConfig<DX, MSUB>;
    static_assert(DX || !DROP, "only the input gradient masks its accumulator");
    constexpr int LS = C::kLS, DS = C::kDS;
    constexpr int kWork = C::kWorkWarps * 32;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ uint64_t bar_full[LS], bar_empty[LS], bar_dfull[DS], bar_dempty[DS], bar_accum, bar_ext, bar_masked;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // the offsets, the activations and the encoded weight were complete before
    // the kernel this one depends on released it (that kernel waited for all
    // earlier ones first); T2 / V2 is that kernel's and is waited for below
    GroupTile g;
    const int ct = args.cols_fastest ? blockIdx.x : blockIdx.y;
    const int rt = args.cols_fastest ? blockIdx.y : blockIdx.x;
    if (!find_tile(args.offsets, args.E, args.M, C::kRows, rt, lane, g)) {
        // every CTA waits, so this grid's completion implies the earlier kernels'
        grid_dependency_wait();
        return;
    }
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* base = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    auto a_buf = [&](int it) { return base + (it % LS) * C::kLoadSlot; };
    auto codes_buf = [&](int it) { return base + (it % LS) * C::kLoadSlot + C::kABytes; };
    auto b_buf = [&](int it) { return base + LS * C::kLoadSlot + (it % DS) * C::kBBytes; };
    const int c0 = ct * C::kBN;
    const int n_main = args.k_main, n_ext = args.k_ext, n_iter = n_main + n_ext;
    // iteration it: the extension steps come last, or first with dropout
    auto is_main = [&](int it) { return DROP ? it >= n_ext : it < n_main; };
    const int main0 = DROP ? n_ext : 0, ext0 = DROP ? 0 : n_main;
    const int nsub = MSUB == 2 && g.row_end - g.row0 <= C::kBM ? 1 : MSUB;

    if (threadIdx.x == 0) {
        for (int i = 0; i < LS; ++i) {
            mbar_init(&bar_full[i], 1);
            mbar_init(&bar_empty[i], 1);
        }
        for (int i = 0; i < DS; ++i) {
            mbar_init(&bar_dfull[i], C::kTeamWarps);
            mbar_init(&bar_dempty[i], 1);
        }
        mbar_init(&bar_accum, 1);
        mbar_init(&bar_ext, 1);
        mbar_init(&bar_masked, C::kWorkWarps);
        s_abort = 0;
        fence_barrier_init();
    }
    // thread 0 goes straight on to the copies (see k_gemm)
    if (threadIdx.x == 0) asm volatile("barrier.arrive 3, %0;" ::"r"(C::kThreads) : "memory");
    else asm volatile("barrier.sync 3, %0;" ::"r"(C::kThreads) : "memory");
    volatile int* abort_flag = &s_abort;

    if (warp == 0) {
        // ------------------------------------------------------------ copies
        if (lane == 0) {
            tma_prefetch_desc(&map_a);
            tma_prefetch_desc(&map_w);
            tma_prefetch_desc(&map_ae);
            tma_prefetch_desc(&map_be);
            int issued = 0;
            for (int it = 0; it < n_iter; ++it) {
                if (it >= LS && !mbar_wait(&bar_empty[it % LS], ((it / LS) & 1u) ^ 1u, abort_flag)) break;
                if (*abort_flag) break;
                uint64_t* bar = &bar_full[it % LS];
                if (is_main(it)) {
                    const int kb = it - main0;
                    mbar_arrive_expect_tx(bar, nsub * C::kSub + C::kCBytes);
                    for (int ms = 0; ms < nsub; ++ms)
                        tma_load_2d(a_buf(it) + ms * C::kSub, &map_a, bar, kb * 64, g.row0 + ms * C::kBM);
                    if constexpr (DX) tma_load_3d(codes_buf(it), &map_w, bar, c0 / 2, kb * 64, g.e);
                    else tma_load_3d(codes_buf(it), &map_w, bar, kb * 32, c0, g.e);
                } else {
                    const int j = it - ext0;
                    // the factor's tile lands in a decode slot
                    if (it >= DS && !mbar_wait(&bar_dempty[it % DS], ((it / DS) & 1u) ^ 1u, abort_flag)) break;
                    if (j == 0) grid_dependency_wait();
                    const int jb = j % (n_ext / 2);  // [hi | lo] against the factor twice
                    mbar_arrive_expect_tx(bar, nsub * C::kSub + C::kBBytes);
                    for (int ms = 0; ms < nsub; ++ms)
                        tma_load_2d(a_buf(it) + ms * C::kSub, &map_ae, bar, j * 64, g.row0 + ms * C::kBM);
                    if constexpr (DX) {
#pragma unroll
                        for (int c = 0; c < C::kBN / 64; ++c)
                            tma_load_3d(b_buf(it) + c * 8192, &map_be, bar, c0 + c * 64, jb * 64, g.e);
                    } else {
                        tma_load_3d(b_buf(it), &map_be, bar, jb * 64, c0, g.e);
                    }
                }
                ++issued;
            }
            if (*abort_flag) {
                // let the copies already issued land before the CTA exits
                for (int it = issued > LS ? issued - LS : 0; it < issued; ++it)
                    mbar_drain(&bar_full[it % LS], (it / LS) & 1u);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ tensor memory, MMAs
        tmem_alloc(&s_tmem, C::kTmemCols);
        tmem_relinquish();
        tc_fence_before();
        asm volatile("bar.arrive 2, %0;" ::"r"(32 + kWork) : "memory");
        __syncwarp();
        tc_fence_after();
        const uint32_t tmem_d = s_tmem;
        if (lane == 0) {
            for (int it = 0; it < n_iter; ++it) {
                if (!mbar_wait(&bar_full[it % LS], (it / LS) & 1u, abort_flag)) break;
                if (is_main(it)) {
                    // fills of this decode slot by the decoders so far (with
                    // dropout its first uses held extension tiles)
                    const int slot = it % DS;
                    int fills = it / DS;
                    if (DROP && n_ext > slot) fills -= (n_ext - slot + DS - 1) / DS;
                    if (!mbar_wait(&bar_dfull[slot], fills & 1u, abort_flag)) break;
                    if (DROP && it == main0 && !mbar_wait(&bar_masked, 0, abort_flag)) break;
                }
                tc_fence_after();
                const uint32_t a_base = smem_u32(a_buf(it)), b_base = smem_u32(b_buf(it));
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const uint64_t bdesc = tile_desc(b_base, DX, kk);
                    for (int ms = 0; ms < nsub; ++ms)
                        mma_bf16_ss(tmem_d + ms * C::kBN, tile_desc(a_base + ms * C::kSub, false, kk), bdesc,
                                    C::kIdesc, it * 4 + kk > 0 ? 1u : 0u);
                }
                mma_commit(&bar_empty[it % LS]);
                mma_commit(&bar_dempty[it % DS]);
                if (DROP && it == n_ext - 1) mma_commit(&bar_ext);
            }
            mma_commit(&bar_accum);
        }
    } else {
        const int ew = warp - 2;
        const int q = warp & 3;  // tensor memory lane quadrant of this warp
        constexpr int cw = C::kBN / (C::kWorkWarps / 4);
        const int cbeg = (ew / 4) * cw;
        uint32_t tmem_d = 0;
        if constexpr (DROP) {
            // -------------------------------------------------------- keep and scale V A
            asm volatile("bar.sync 2, %0;" ::"r"(32 + kWork) : "memory");
            tc_fence_after();
            tmem_d = s_tmem;
            KeepGen gen;
            grid_dependency_wait();  // the generator's state may be as young as V
            gen.init(args.drop);
            if (mbar_wait(&bar_ext, 0, abort_flag)) {
                tc_fence_after();
                for (int ms = 0; ms < nsub; ++ms) {
                    const int64_t row = g.row0 + ms * C::kBM + q * 32 + lane;
#pragma unroll 1
                    for (int cc = cbeg; cc < cbeg + cw; cc += 32) {
                        const uint32_t at = tmem_d + (static_cast<uint32_t>(q * 32) << 16) + ms * C::kBN + cc;
                        uint32_t v[32];
                        tmem_ld_32x32b_x32(at, v);
                        tmem_ld_wait();
                        const uint64_t grp = static_cast<uint64_t>(row * args.cols + c0 + cc) >> 3;
#pragma unroll
                        for (int o = 0; o < 4; ++o) {
                            uint32_t f[4];
                            gen.flags(grp + o, f);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                uint32_t& x = v[8 * o + 2 * i];
                                uint32_t& y = v[8 * o + 2 * i + 1];
                                x = (f[i] & 0x8000u) ? __float_as_uint(__uint_as_float(x) * args.drop.gain) : 0u;
                                y = (f[i] >> 31) ? __float_as_uint(__uint_as_float(y) * args.drop.gain) : 0u;
                            }
                        }
                        tmem_st_32x32b_x32(at, v);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_masked);
        }
        // ------------------------------------------------------------ decoders
        {
            const int team = ew / C::kTeamWarps;
            const int dt = threadIdx.x - 64 - team * C::kTeamThreads;
            const bool fp32_scales = args.absmax != nullptr;  // no double quantisation
            const float mu = fp32_scales ? 0.0f : __ldg(args.scale_mean);
            // This thread's unit of a step.  Forward: weight row c0 + dt, block
            // kb.  Input gradient: weight row 64 kb + n_local, block cblk of the
            // tile, dealt so that stores and code reads meet few bank conflicts
            // (see k_gemm).
            constexpr int kCB = C::kBN / 64;
            int n_local = dt, cblk = 0;
            if constexpr (DX) {
                const int qw = dt >> 3, i = dt & 7;
                n_local = 8 * (qw / kCB) + i;
                cblk = (i + qw % kCB) % kCB;
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
                const int wrow = DX ? kb * 64 + n_local : c0 + dt;
                const int wblk = DX ? c0 / 64 + cblk : kb;
                ok_pf[slot] = kb < n_main && wrow < args.w_rows && wblk < args.w_blocks_per_row;
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
            for (int u = 0; u < kPf; ++u) fetch(team + u * C::kTeams, u);
            bool stop = false;
            for (int kb0 = team; kb0 < n_main && !stop; kb0 += kPf * C::kTeams) {
#pragma unroll
                for (int u = 0; u < kPf; ++u) {
                    const int kb = kb0 + u * C::kTeams;
                    if (kb >= n_main) break;
                    const int it = kb + main0;
                    const bool valid = ok_pf[u];
                    const float sc =
                        valid ? (fp32_scales ? a2_pf[u] : nf4_block_scale(q_pf[u], a2_pf[u], mu)) : 0.0f;
                    fetch(kb + kPf * C::kTeams, u);
                    if (!mbar_wait(&bar_full[it % LS], (it / LS) & 1u, abort_flag) ||
                        (it >= DS && !mbar_wait(&bar_dempty[it % DS], ((it / DS) & 1u) ^ 1u, abort_flag))) {
                        stop = true;
                        break;
                    }
                    uint8_t* dst = b_buf(it) + dst_off;
                    if (!valid) zero_row(dst);
                    else decode_unit_reg(codes_buf(it) + code_off, sc, dst, swz);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar_dfull[it % DS]);
                }
            }
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
            for (int ms = 0; ms < nsub; ++ms) {
                const int row = g.row0 + ms * C::kBM + q * 32 + lane;
                const bool row_ok = row < g.row_end;
                for (int cc = cbeg; cc < cbeg + cw; cc += 32) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(tmem_d + (static_cast<uint32_t>(q * 32) << 16) + ms * C::kBN + cc, v);
                    tmem_ld_wait();
                    if (row_ok) {
                        uint16_t* dst = args.out + static_cast<int64_t>(row) * args.cols + c0 + cc;
#pragma unroll
                        for (int j = 0; j < 32; j += 8) {
                            if (c0 + cc + j < args.cols) {  // cols is a multiple of 8
                                uint4 pk;
                                pk.x = pack_bf16x2(__uint_as_float(v[j]), __uint_as_float(v[j + 1]));
                                pk.y = pack_bf16x2(__uint_as_float(v[j + 2]), __uint_as_float(v[j + 3]));
                                pk.z = pack_bf16x2(__uint_as_float(v[j + 4]), __uint_as_float(v[j + 5]));
                                pk.w = pack_bf16x2(__uint_as_float(v[j + 6]), __uint_as_float(v[j + 7]));
                                *reinterpret_cast<uint4*>(dst + j) = pk;
                            }
                        }
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(s_tmem, C::kTmemCols);
    }
}

}  // namespace nf4lora
