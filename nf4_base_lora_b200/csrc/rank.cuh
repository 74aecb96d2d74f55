// The rank-r products of the adapter over ragged row groups, with dropout on
// the adapter's input, on tcgen05:
//
//   RANK_T   T_i  = s gain (keep_i .* X_i) A_e^T       rows i of group e
//   RANK_V   V_i  = s dY_i B_e
//   RANK_DB  dB_e = sum_i dY_i^T T_i                   [N, r]
//   RANK_DA  dA_e = gain sum_i V_i^T (keep_i .* X_i)   [r, K]
//
// All four read one large activation once and are bound by that stream (HBM);
// the MMAs are N = r wide and idle most of the time.  T and V split the
// contraction over grid.z into fp32 partials that k_rank_rows_sum adds in a
// fixed order; dB and dA contract over a group's rows, 256 output rows per CTA
// (two accumulators sharing the narrow operand), and write their result
// themselves where the experts alone fill the SMs.  T and V enter dB and dA as
// their 16-bit pair [hi | lo], both halves into the same accumulator columns.
//
// Dropout: the activation tile has landed in shared memory in the swizzled
// operand layout, whose 16-byte pieces are exactly the generator's groups of
// eight elements; eight warps clear the dropped elements of each piece in place
// (the gain goes into the product's factor, so no kept element is rounded) and
// hand the tile to the MMAs.  The last step of a group that does not end on a
// step's 64 rows gets the rows behind its end cleared the same way, in both
// operands: they belong to the next group, or to nobody and may hold anything.
//
// Warp roles: warp 0 copies, warp 1 owns tensor memory and issues the MMAs,
// warps 2 .. 9 clear elements and run the epilogue.
#pragma once

#include <cstdint>

#include "gemm.cuh"
#include "grouped.cuh"
#include "philox.cuh"

namespace nf4lora {

enum RankMode : int { RANK_T = 0, RANK_V = 1, RANK_DB = 2, RANK_DA = 3 };

struct RankArgs {
    const int32_t* offsets;
    int E;
    int M;
    int rows;          // dB: N, dA: K (output rows per expert)
    int k_steps;       // T, V: 64-wide steps of the contraction
    int k_per_split;   // T, V
    int splits;        // dB, dA: parts of a group's rows
    int r, rn;         // rank; MMA width, r rounded up to 16
    int r64;           // column of the low halves in T2 / V2
    int stages, a_bytes, b_bytes;
    int tmem_cols;
    DropArgs drop;
    int drop_cols;     // K
    float alpha;       // dB, dA written here
    float* part;       // T, V: [split][M][rn]; dB: [split][E][N][rn]; dA: [split][E][rn][K]
    int64_t part_slice;
    uint16_t* out;     // dB [E][N][r] / dA [E][r][K] written here, or NULL (partials)
    int accumulate;
};

constexpr int kRankStages = 8;  // at most
constexpr int kRankWarps = 8;
constexpr int kRankThreads = 64 + 32 * kRankWarps;

__device__ __forceinline__ uint16_t bf16_bits(float v) {
    const __nv_bfloat16 h = __float2bfloat16_rn(v);
    return *reinterpret_cast<const uint16_t*>(&h);
}

// map_a: the activation; T, V: box {64, 128} (K-major), dB, dA: box {64, 64}
// (MN-major).  map_b: T: A (K, r, E), box {64, rn, 1}; V: B (r, N, E), box
// {64, 64, 1}; dB, dA: T2 / V2 [M, 2 r64], box {64, 64}.
template <int MODE, bool DROP>
__global__ void __launch_bounds__(kRankThreads, 2)
    k_rank(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const RankArgs args) {
    constexpr bool TOK = MODE == RANK_DB || MODE == RANK_DA;  // contraction over a group's rows
    static_assert(!DROP || MODE == RANK_T || MODE == RANK_DA, "only X is dropped");
    constexpr int kOutRows = TOK ? 256 : 128;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ uint64_t bar_full[kRankStages], bar_empty[kRankStages], bar_clear[kRankStages], bar_last, bar_tail, bar_accum;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // it overwrites what the kernels before it may still read (the partials)
    grid_dependency_wait();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    GroupTile g;
    int out0 = 0, begin = 0, n_steps, step0;
    if constexpr (!TOK) {
        if (!find_tile<false>(args.offsets, args.E, args.M, 128, blockIdx.x, lane, g)) return;
        step0 = blockIdx.z * args.k_per_split;
        n_steps = min(args.k_per_split, args.k_steps - step0);
    } else {
        g.e = blockIdx.y;
        g.row_end = args.M;
        if (args.offsets != nullptr) group_bounds(args.offsets, g.e, args.M, begin, g.row_end);
        out0 = blockIdx.x * kOutRows;
        const int total = (g.row_end - begin + 63) / 64;
        const int per = (total + args.splits - 1) / args.splits;
        step0 = blockIdx.z * per;
        n_steps = max(0, min(per, total - step0));
    }
    const int LS = args.stages, slot_bytes = args.a_bytes + args.b_bytes;
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* base = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    auto a_buf = [&](int it) { return base + (it % LS) * slot_bytes; };
    auto b_buf = [&](int it) { return base + (it % LS) * slot_bytes + args.a_bytes; };
    const int rchunks = (args.rn + 63) / 64;
    // rows of the group in the step after which it ends (64: no partial step here)
    int tail_rows = 64;
    if (TOK && n_steps > 0) tail_rows = min(64, g.row_end - (begin + 64 * (step0 + n_steps - 1)));
    // dense calls end where the array does, whose copies read zeros behind it
    const bool has_tail = TOK && args.offsets != nullptr && tail_rows < 64;

    // The barrier on which step `it` lands, and its parity.  Without dropout the
    // clearing warps look at the last step alone; a wait on the ring's barrier
    // could not tell its phases apart there, so that step has a barrier of its own.
    auto own_bar = [&](int it) { return !DROP && has_tail && it == n_steps - 1; };
    auto full_bar = [&](int it) { return own_bar(it) ? &bar_last : &bar_full[it % LS]; };
    auto full_parity = [&](int it) { return own_bar(it) ? 0u : (it / LS) & 1u; };

    if (threadIdx.x == 0) {
        for (int i = 0; i < LS; ++i) {
            mbar_init(&bar_full[i], 1);
            mbar_init(&bar_empty[i], 1);
            mbar_init(&bar_clear[i], kRankWarps);
        }
        mbar_init(&bar_last, 1);
        mbar_init(&bar_tail, kRankWarps);
        mbar_init(&bar_accum, 1);
        s_abort = 0;
        fence_barrier_init();
    }
    __syncthreads();
    volatile int* abort_flag = &s_abort;

    if (warp == 0) {
        if (lane == 0) {
            tma_prefetch_desc(&map_a);
            tma_prefetch_desc(&map_b);
            int issued = 0;
            for (int it = 0; it < n_steps; ++it) {
                if (it >= LS && !mbar_wait(&bar_empty[it % LS], ((it / LS) & 1u) ^ 1u, abort_flag)) break;
                if (*abort_flag) break;
                uint64_t* bar = full_bar(it);
                const int k = 64 * (step0 + it);
                mbar_arrive_expect_tx(bar, slot_bytes);
                if constexpr (!TOK) {
                    tma_load_2d(a_buf(it), &map_a, bar, k, g.row0);
                    if constexpr (MODE == RANK_T) {
                        tma_load_3d(b_buf(it), &map_b, bar, k, 0, g.e);
                    } else {
                        for (int c = 0; c < rchunks; ++c)
                            tma_load_3d(b_buf(it) + c * 8192, &map_b, bar, 64 * c, k, g.e);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < kOutRows / 64; ++c)
                        tma_load_2d(a_buf(it) + c * 8192, &map_a, bar, out0 + 64 * c, begin + k);
                    for (int c = 0; c < rchunks; ++c) {
                        tma_load_2d(b_buf(it) + c * 8192, &map_b, bar, 64 * c, begin + k);
                        tma_load_2d(b_buf(it) + (rchunks + c) * 8192, &map_b, bar, args.r64 + 64 * c, begin + k);
                    }
                }
                ++issued;
            }
            if (*abort_flag)
                for (int it = issued > LS ? issued - LS : 0; it < issued; ++it)
                    mbar_drain(full_bar(it), full_parity(it));
        }
    } else if (warp == 1) {
        tmem_alloc(&s_tmem, args.tmem_cols);
        tmem_relinquish();
        tc_fence_before();
        asm volatile("bar.arrive 2, %0;" ::"r"(32 + 32 * kRankWarps) : "memory");
        __syncwarp();
        tc_fence_after();
        const uint32_t tmem_d = s_tmem;
        const uint32_t idesc = make_idesc_bf16(128, 0, TOK ? 1 : 0, MODE == RANK_T ? 0 : 1) |
                               (static_cast<uint32_t>(args.rn >> 3) << 17);
        if (lane == 0) {
            for (int it = 0; it < n_steps; ++it) {
                if (!mbar_wait(full_bar(it), full_parity(it), abort_flag)) break;
                if (DROP) {
                    if (!mbar_wait(&bar_clear[it % LS], (it / LS) & 1u, abort_flag)) break;
                } else if (has_tail && it == n_steps - 1) {
                    if (!mbar_wait(&bar_tail, 0, abort_flag)) break;
                }
                tc_fence_after();
                const uint32_t a_base = smem_u32(a_buf(it)), b_base = smem_u32(b_buf(it));
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const uint32_t first = it * 4 + kk > 0 ? 1u : 0u;
                    if constexpr (!TOK) {
                        mma_bf16_ss(tmem_d, tile_desc(a_base, false, kk), tile_desc(b_base, MODE == RANK_V, kk), idesc,
                                    first);
                    } else {
                        const uint64_t hi = tile_desc(b_base, true, kk);
                        const uint64_t lo = tile_desc(b_base + rchunks * 8192, true, kk);
#pragma unroll
                        for (int ms = 0; ms < 2; ++ms) {
                            const uint64_t a = tile_desc(a_base + ms * 16384, true, kk);
                            mma_bf16_ss(tmem_d + ms * args.rn, a, hi, idesc, first);
                            mma_bf16_ss(tmem_d + ms * args.rn, a, lo, idesc, 1u);
                        }
                    }
                }
                mma_commit(&bar_empty[it % LS]);
            }
            mma_commit(&bar_accum);
        }
    } else {
        const int ew = warp - 2, wt = threadIdx.x - 64;
        // ------------------------------------------------------------ clearing
        if (DROP || has_tail) {
            KeepGen gen;
            if constexpr (DROP) gen.init(args.drop);
            for (int it = DROP ? 0 : n_steps - 1; it < n_steps; ++it) {
                if (!mbar_wait(full_bar(it), full_parity(it), abort_flag)) break;
                uint8_t* a = a_buf(it);
                const int k = 64 * (step0 + it);
                if constexpr (DROP) {
                    constexpr int kPieces = kOutRows * 8 / (32 * kRankWarps);  // 16-byte pieces per thread
#pragma unroll
                    for (int i = 0; i < kPieces; ++i) {
                        const int p = wt + i * 32 * kRankWarps;
                        const int c = p & 7;
                        int off;
                        int64_t elem;  // flat index in X of the piece's first element
                        if constexpr (!TOK) {
                            const int row = p >> 3;
                            off = row * 128 + ((c ^ (row & 7)) << 4);
                            elem = static_cast<int64_t>(g.row0 + row) * args.drop_cols + k + 8 * c;
                        } else {
                            const int chunk = p >> 9, row = (p >> 3) & 63;
                            off = chunk * 8192 + row * 128 + ((c ^ (row & 7)) << 4);
                            elem = static_cast<int64_t>(begin + k + row) * args.drop_cols + out0 + 64 * chunk + 8 * c;
                        }
                        uint4* at = reinterpret_cast<uint4*>(a + off);
                        uint4 v = *at;
                        uint32_t m[4];
                        gen.masks(static_cast<uint64_t>(elem) >> 3, m);
                        v.x &= m[0];
                        v.y &= m[1];
                        v.z &= m[2];
                        v.w &= m[3];
                        *at = v;
                    }
                }
                if (TOK && has_tail && it == n_steps - 1) {
                    // rows behind the group's end: whole 128-byte rows of every chunk
                    if (DROP) named_barrier_sync(4, 32 * kRankWarps);  // the pieces above are other threads'
                    const int chunks = kOutRows / 64 + 2 * rchunks, per = (64 - tail_rows) * 8;
                    for (int p = wt; p < chunks * per; p += 32 * kRankWarps) {
                        const int chunk = p / per, rem = p - chunk * per;
                        uint8_t* src = chunk < kOutRows / 64 ? a + chunk * 8192
                                                             : b_buf(it) + (chunk - kOutRows / 64) * 8192;
                        *reinterpret_cast<uint4*>(src + tail_rows * 128 + rem * 16) = make_uint4(0, 0, 0, 0);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(DROP ? &bar_clear[it % LS] : &bar_tail);
            }
        }
        // ------------------------------------------------------------ epilogue
        asm volatile("bar.sync 2, %0;" ::"r"(32 + 32 * kRankWarps) : "memory");
        tc_fence_after();
        const uint32_t tmem_d = s_tmem;
        const int q = warp & 3, half = ew >> 2;
        const bool ok = mbar_wait(&bar_accum, 0, abort_flag) && !*abort_flag;
        tc_fence_after();
        if (ok && (n_steps > 0 || TOK)) {
            // T, V: the two halves of the warps share the columns; dB, dA: they
            // take one accumulator each
            const int cols = TOK ? args.rn : args.rn / 2;
            const int cbeg = TOK ? 0 : half * cols;
            const int lrow = q * 32 + lane + (TOK ? half * 128 : 0);
            const int row = TOK ? out0 + lrow : g.row0 + lrow;
            const bool row_ok = row < (TOK ? args.rows : g.row_end);
            const uint32_t at = tmem_d + (static_cast<uint32_t>(q * 32) << 16) + (TOK ? half * args.rn : 0);
            for (int cc = cbeg; cc < cbeg + cols; cc += 8) {
                uint32_t v[8];
                if (n_steps > 0) {
                    tmem_ld_32x32b_x8(at + cc, v);
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = 0u;  // a group without rows
                }
                if (!row_ok) continue;
                if constexpr (!TOK) {
                    float* dst = args.part + blockIdx.z * args.part_slice + static_cast<int64_t>(row) * args.rn + cc;
                    *reinterpret_cast<uint4*>(dst) = make_uint4(v[0], v[1], v[2], v[3]);
                    *reinterpret_cast<uint4*>(dst + 4) = make_uint4(v[4], v[5], v[6], v[7]);
                } else if constexpr (MODE == RANK_DB) {
                    if (args.out == nullptr) {
                        float* dst = args.part + blockIdx.z * args.part_slice +
                                     (static_cast<int64_t>(g.e) * args.rows + row) * args.rn + cc;
                        *reinterpret_cast<uint4*>(dst) = make_uint4(v[0], v[1], v[2], v[3]);
                        *reinterpret_cast<uint4*>(dst + 4) = make_uint4(v[4], v[5], v[6], v[7]);
                    } else {
                        uint16_t* dst = args.out + (static_cast<int64_t>(g.e) * args.rows + row) * args.r + cc;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (cc + j < args.r) {
                                float x = __uint_as_float(v[j]) * args.alpha;
                                if (args.accumulate) x += bf16_bits_to_float(dst[j]);
                                dst[j] = bf16_bits(x);
                            }
                    }
                } else {
                    if (args.out == nullptr) {
                        float* dst = args.part + blockIdx.z * args.part_slice +
                                     (static_cast<int64_t>(g.e) * args.rn + cc) * args.rows + row;
#pragma unroll
                        for (int j = 0; j < 8; ++j) dst[static_cast<int64_t>(j) * args.rows] = __uint_as_float(v[j]);
                    } else {
                        uint16_t* dst = args.out + (static_cast<int64_t>(g.e) * args.r + cc) * args.rows + row;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (cc + j < args.r) {
                                uint16_t* d = dst + static_cast<int64_t>(j) * args.rows;
                                float x = __uint_as_float(v[j]) * args.alpha;
                                if (args.accumulate) x += bf16_bits_to_float(*d);
                                *d = bf16_bits(x);
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
        tmem_dealloc(s_tmem, args.tmem_cols);
    }
}

// ------------------------------------------------------------------ sums of the splits
// T2 / V2 [M, 2 r64] = 16-bit pair of alpha sum_z part[z], zero beyond r; T also
// as fp32 [M, r].  Rows outside the groups are left as they are.
struct RankRowsSumArgs {
    const int32_t* offsets;
    int E;
    int M;
    const float* part;
    int splits;
    int64_t slice;
    int r, rn, r64;
    float alpha;
    uint16_t* pair;
    float* out32;  // or NULL
    int check;     // 1: report offsets that break the contract in the device status word
};

__global__ void k_rank_rows_sum(const RankRowsSumArgs a) {
    grid_dependency_wait();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int lo = 0, hi = a.M;
    if (a.offsets != nullptr) {
        lo = min(max(__ldcg(a.offsets), 0), a.M);
        hi = min(max(__ldcg(a.offsets + a.E), lo), a.M);
        if (a.check && blockIdx.x == 0) {
            bool bad = false;
            for (int e = threadIdx.x; e <= a.E; e += blockDim.x) {
                const int v = __ldcg(a.offsets + e);
                bad |= v < (e > 0 ? max(0, __ldcg(a.offsets + e - 1)) : 0) || v > a.M;
            }
            if (bad) atomicCAS(&g_device_status, 0, kStatusOffsets);
        }
    }
    const int quads = a.r64 / 4;
    const int64_t total = static_cast<int64_t>(hi - lo) * quads;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t row = lo + i / quads;
        const int j = 4 * static_cast<int>(i % quads);
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (j < a.rn) {
            const float* p = a.part + row * a.rn + j;
            for (int z = 0; z < a.splits; ++z) {
                const float4 x = __ldcg(reinterpret_cast<const float4*>(p + z * a.slice));
                v[0] += x.x;
                v[1] += x.y;
                v[2] += x.z;
                v[3] += x.w;
            }
        }
        float hi4[4], lo4[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            v[u] = j + u < a.r ? v[u] * a.alpha : 0.0f;
            hi4[u] = __bfloat162float(__float2bfloat16_rn(v[u]));
            lo4[u] = v[u] - hi4[u];
            if (a.out32 != nullptr && j + u < a.r) a.out32[row * a.r + j + u] = v[u];
        }
        uint16_t* dst = a.pair + row * 2 * a.r64 + j;
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(hi4[0], hi4[1]), pack_bf16x2(hi4[2], hi4[3]));
        *reinterpret_cast<uint2*>(dst + a.r64) = make_uint2(pack_bf16x2(lo4[0], lo4[1]), pack_bf16x2(lo4[2], lo4[3]));
    }
}

// The pair of a saved fp32 T [M, r].
__global__ void k_rank_pair(const float* __restrict__ src, int64_t M, int r, int r64, uint16_t* __restrict__ pair) {
    grid_dependency_wait();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t total = M * r64;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t m = i / r64;
        const int j = static_cast<int>(i % r64);
        const float v = j < r ? src[m * r + j] : 0.0f;
        const __nv_bfloat16 hi = __float2bfloat16_rn(v);
        pair[m * 2 * r64 + j] = *reinterpret_cast<const uint16_t*>(&hi);
        pair[m * 2 * r64 + r64 + j] = bf16_bits(v - __bfloat162float(hi));
    }
}

// dB [E][N][r] (TRANSPOSED false) or dA [E][r][K] from partials
// [split][E][N][rn] or [split][E][rn][K], the splits added in order.
template <bool TRANSPOSED>
__global__ void k_rank_grad_sum(const float* __restrict__ part, int splits, int64_t slice, int64_t E, int rows, int r,
                                int rn, float alpha, uint16_t* __restrict__ out, int accumulate) {
    grid_dependency_wait();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t total = E * rows * r;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t inner = TRANSPOSED ? rows : r;
        const int64_t outer = i / inner, c = i - outer * inner;
        int64_t at;
        if (TRANSPOSED) {
            const int64_t e = outer / r, j = outer - e * r;
            at = (e * rn + j) * rows + c;
        } else {
            at = outer * rn + c;
        }
        float v = 0.0f;
        for (int z = 0; z < splits; ++z) v += __ldcg(part + z * slice + at);
        v *= alpha;
        if (accumulate) v += bf16_bits_to_float(out[i]);
        out[i] = bf16_bits(v);
    }
}

}  // namespace nf4lora
