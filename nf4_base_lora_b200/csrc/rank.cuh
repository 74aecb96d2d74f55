// The rank-r products of the adapter over ragged row groups, with dropout on
// the adapter's input, on tcgen05:
//
//   RANK_T   T_i  = s gain (keep_i .* X_i) A_e^T       rows i of group e
//   RANK_V   V_i  = s dY_i B_e
//   RANK_DB  dB_e = sum_i dY_i^T T_i                   [N, r]
//   RANK_DA  dA_e = gain sum_i V_i^T (keep_i .* X_i)   [r, K]
//
// T and V are sums over a whole layer's width that are kept in 32 bits, while the
// tensor cores truncate at every addition: an accumulator takes 16 steps (1024
// products) at most, then the next set of columns, and the sets are added rounded
// (2048 wide: an error of 1e-6 of T's norm and not 2e-6).
//
// All four read one large activation once and are bound by that stream (HBM),
// with dropout by the generator beside it; the MMAs are N = r wide and idle most of
// the time.  8192 tokens over eight experts of 4096 -> 11008, r 16, dropout 0.05: V
// 43 us and dB 42 us for 180 MB of dY (4.2 TB/s), T 23 us and dA 30 us for 67 MB of
// X (2.9 and 2.2 TB/s).  T and V split the
// contraction over grid.z into fp32 partials that k_rank_rows_sum adds in a
// fixed order.  dB and dA contract over a group's rows, 256 output rows per CTA
// (two accumulators sharing the narrow operand); a long group is cut into parts
// of at most part_steps steps, whose partials k_rank_grad_sum adds in order,
// while a group of one part writes its result itself -- so a skewed batch does
// not wait for its longest group, short groups cost no partials, and no
// accumulator takes more than 128 steps of truncating additions.  T and V
// enter dB and dA as their 16-bit pair [hi | lo], both halves into the same
// accumulator columns.
//
// Dropout: the activation tile has landed in shared memory in the swizzled
// operand layout, whose 16-byte pieces are exactly the generator's groups of
// eight elements; the clearing warps zero the dropped elements of each piece in
// place (the gain goes into the product's factor, so no kept element is rounded)
// and hand the tile to the MMAs.  The last step of a group that does not end on a
// step's 64 rows gets the rows behind its end cleared the same way, in both
// operands: they belong to the next group, or to nobody and may hold anything.
//
// Warp roles: warp 0 copies, warp 1 owns tensor memory and issues the MMAs,
// warps 2 .. 9 clear elements and run the epilogue.  Two CTAs share an SM wherever
// two stages of each fit: their starts, which take as long as several steps, and
// their ends overlap.
#pragma once

#include <cstdint>

#include "adapter.h"
#include "gemm.cuh"
#include "grouped.cuh"
#include "philox.cuh"

namespace nf4lora {

enum RankMode : int { RANK_T = 0, RANK_V = 1, RANK_DB = 2, RANK_DA = 3 };

struct RankArgs {
    const int32_t* offsets;
    int check;         // the first kernel of a call that reads the offsets: looks whether they keep their rule
    int E;
    int M;
    int rows;          // dB: N, dA: K (output rows per expert)
    int k_steps;       // T, V: 64-wide steps of the contraction
    int k_per_split;   // T, V
    int run_steps;     // T, V: steps into one set of accumulators
    int part_steps;    // dB, dA
    int slots;         // partials there is room for
    int r, rn;         // rank; MMA width, r rounded up to 16
    int r64;           // column of the low halves in T2 / V2
    int stages, a_bytes, b_bytes;
    int tmem_cols;
    DropArgs drop;
    int drop_cols;     // K
    float alpha;       // dB, dA written here
    float* part;       // T, V: [split][M][rn]; dB: [part][N][rn]; dA: [part][rn][K]
    int64_t part_slice;
    uint16_t* out;     // dB [E][N][r] / dA [E][r][K]
    int accumulate;
    int late_wait;     // dB, dA: the inputs are complete at the start
    uint16_t* pair;    // T, V in one split: the pair [M, 2 r64] and (or NULL) fp32 [M, r], else partials
    float* out32;
};

// v[0 .. 7] = columns j .. j + 7 of a row of T or V: the 16-bit pair, zero beyond
// r, and the fp32 value; the arrays have M rows.
__device__ __forceinline__ void store_pair(float (&v)[8], int64_t row, int j, int64_t M, int r, int r64,
                                           uint16_t* pair, float* out32) {
    float hi[8], lo[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        if (j + u >= r) v[u] = 0.0f;
        hi[u] = bf16_high_part(v[u]);
        lo[u] = v[u] - hi[u];
        if (out32 != nullptr && j + u < r && NF4_CHECK(in_span(out32 + row * r + j + u, 4, out32, M * r * 4, 4), 20))
            out32[row * r + j + u] = v[u];
    }
    uint16_t* dst = pair + row * 2 * r64 + j;
    if (!NF4_CHECK(in_span(dst, 16, pair, M * 4 * r64, 16) && in_span(dst + r64, 16, pair, M * 4 * r64, 16), 21))
        return;
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(hi[0], hi[1]), pack_bf16x2(hi[2], hi[3]),
                                                pack_bf16x2(hi[4], hi[5]), pack_bf16x2(hi[6], hi[7]));
    *reinterpret_cast<uint4*>(dst + r64) = make_uint4(pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3]),
                                                      pack_bf16x2(lo[4], lo[5]), pack_bf16x2(lo[6], lo[7]));
}

constexpr int kRankStages = 8;  // at most
template <int MODE, bool DROP>
struct RankConfig {
    static constexpr bool kTok = MODE == RANK_DB || MODE == RANK_DA;
    static constexpr int kWarps = 8;  // clearing and epilogue
    static constexpr int kThreads = 64 + 32 * kWarps;
};

// The parts of the groups' rows for dB and dA, numbered in group order: a group
// has ceil(rows / (64 part_steps)) of them, at least one.
__device__ __forceinline__ int rank_parts(int n, int part_steps) {
    return max(1, (n + 64 * part_steps - 1) / (64 * part_steps));
}
struct RankPart {
    int e;
    int begin, end;  // the group's rows
    int parts;       // of the group
    int part;        // this one
    int slot;        // of the group's first partial; groups of one part take none
};
// Part u; the whole warp calls it.  False beyond the last.  A group beyond the last slot, which only
// offsets that break their rule can make, stays whole (its later parts are void).
__device__ __forceinline__ bool find_part(const int32_t* offsets, int E, int M, int part_steps, int slots, int u,
                                          int lane, RankPart& p) {
    p.slot = 0;
    if (offsets == nullptr) {
        p.e = 0;
        p.begin = 0;
        p.end = M;
        p.parts = rank_parts(M, part_steps);
        p.part = u;
        return p.part < p.parts;
    }
    int before = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
        const int e = e0 + lane;
        int begin = 0, end = 0, n = 0;
        if (e < E) {
            group_bounds(offsets, e, M, begin, end);
            n = rank_parts(end - begin, part_steps);
        }
        const int taken = n > 1 ? n : 0;
        int incl = n, sl = taken;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, incl, d), w = __shfl_up_sync(0xFFFFFFFFu, sl, d);
            if (lane >= d) {
                incl += v;
                sl += w;
            }
        }
        const unsigned hit = __ballot_sync(0xFFFFFFFFu, before + incl > u);
        if (hit != 0) {
            const int src = __ffs(hit) - 1;
            p.e = e0 + src;
            p.begin = __shfl_sync(0xFFFFFFFFu, begin, src);
            p.end = __shfl_sync(0xFFFFFFFFu, end, src);
            p.parts = __shfl_sync(0xFFFFFFFFu, n, src);
            p.part = u - before - __shfl_sync(0xFFFFFFFFu, incl - n, src);
            p.slot += __shfl_sync(0xFFFFFFFFu, sl - taken, src);
            if (p.parts > 1 && p.slot + p.parts > slots) p.parts = 1;
            return p.part < p.parts;
        }
        before += __shfl_sync(0xFFFFFFFFu, incl, 31);
        p.slot += __shfl_sync(0xFFFFFFFFu, sl, 31);
    }
    return false;
}

__device__ __forceinline__ uint16_t bf16_bits(float v) {
    const __nv_bfloat16 h = __float2bfloat16_rn(v);
    return *reinterpret_cast<const uint16_t*>(&h);
}

// map_a: the activation; T, V: box {64, 128} (K-major), dB, dA: box {64, 64}
// (MN-major).  map_b: T: A (K, r, E), box {64, rn, 1}; V: B (r, N, E), box
// {64, 64, 1}; dB, dA: T2 / V2 [M, 2 r64], box {64, 64}.
template <int MODE, bool DROP>
__global__ void __launch_bounds__(RankConfig<MODE, DROP>::kThreads, 2)
    k_rank(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const RankArgs args) {
    using C = RankConfig<MODE, DROP>;
    constexpr bool TOK = C::kTok;  // contraction over a group's rows
    static_assert(!DROP || MODE == RANK_T || MODE == RANK_DA, "only X is dropped");
    constexpr int kOutRows = TOK ? 256 : 128, kWork = 32 * C::kWarps;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ uint64_t bar_full[kRankStages], bar_empty[kRankStages], bar_clear[kRankStages], bar_last, bar_tail,
        bar_accum;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // It overwrites what the kernels before it may still read (the partials).
    // Where all that it reads was complete before the kernel this one depends on
    // released it, only the results wait, and the products run beside that
    // kernel's last CTAs.  Those have all started then, and none can be kept waiting
    // by this kernel's tensor memory: what shares an SM with another CTA has 256
    // columns at most (the input gradient's 32-token kernel 64), and what has more
    // fills an SM's shared memory.
    if (!TOK || !args.late_wait) grid_dependency_wait();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (args.check && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) {
        // offsets that break the contract are reported in the device status word,
        // also where they leave this block, or every block, without rows
        bool bad = false;
        for (int e = threadIdx.x; e <= args.E; e += C::kThreads) {
            const int v = __ldcg(args.offsets + e);
            bad |= v < (e > 0 ? max(0, __ldcg(args.offsets + e - 1)) : 0) || v > args.M;
        }
        if (bad) atomicCAS(&g_device_status, 0, kStatusOffsets);
        __syncwarp();
    }
    GroupTile g;
    int out0 = 0, begin = 0, n_steps, step0;
    RankPart part{0, 0, 0, 1, 0, 0};
    if constexpr (!TOK) {
        if (!find_tile<false>(args.offsets, args.E, args.M, 128, blockIdx.x, lane, g)) return;
        step0 = blockIdx.z * args.k_per_split;
        n_steps = min(args.k_per_split, args.k_steps - step0);
    } else {
        if (!find_part(args.offsets, args.E, args.M, args.part_steps, args.slots, blockIdx.y, lane, part)) {
            grid_dependency_wait();  // this grid's completion implies that of those before it
            return;
        }
        g.e = part.e;
        begin = part.begin;
        g.row_end = part.end;
        out0 = blockIdx.x * kOutRows;
        const int total = (g.row_end - begin + 63) / 64;
        const int per = (total + part.parts - 1) / part.parts;
        step0 = part.part * per;
        n_steps = max(0, min(per, total - step0));
    }
    n_steps = __shfl_sync(0xFFFFFFFFu, n_steps, 0);  // said to be uniform, as what follows from it
    const int LS = args.stages, slot_bytes = args.a_bytes + args.b_bytes;
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* base = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const int rchunks = (args.rn + 63) / 64;
    // rows of the group in the step after which it ends (64: no partial step here)
    int tail_rows = 64;
    if (TOK && n_steps > 0) tail_rows = min(64, g.row_end - (begin + 64 * (step0 + n_steps - 1)));
    // dense calls end where the array does, whose copies read zeros behind it
    const bool has_tail = TOK && args.offsets != nullptr && tail_rows < 64;
    // The barrier on which step `it` lands.  Without dropout the clearing warps
    // look at the last step alone; a wait on the ring's barrier could not tell its
    // phases apart there, so that step has a barrier of its own.
    auto own_bar = [&](int it) { return !DROP && has_tail && it == n_steps - 1; };

    if (threadIdx.x == 0) {
        for (int i = 0; i < LS; ++i) {
            mbar_init(&bar_full[i], 1);
            mbar_init(&bar_empty[i], 1);
            mbar_init(&bar_clear[i], C::kWarps);
        }
        mbar_init(&bar_last, 1);
        mbar_init(&bar_tail, C::kWarps);
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
        }
        __syncwarp();
        int slot = 0;
        uint32_t phase = 1;  // of the slot's release; passes at once in the first round
        bool stop = false;
        for (int it = 0; it < n_steps; ++it) {
            const bool late = it >= LS && !mbar_wait(&bar_empty[slot], phase, abort_flag);
            stop = __any_sync(0xFFFFFFFFu, late || *abort_flag);
            if (stop) break;
            if (elect_one()) {
                uint64_t* bar = own_bar(it) ? &bar_last : &bar_full[slot];
                uint8_t* a_buf = base + slot * slot_bytes;
                uint8_t* b_buf = a_buf + args.a_bytes;
                const int k = 64 * (step0 + it);
                mbar_arrive_expect_tx(bar, slot_bytes);
                if (!NF4_CHECK(in_smem(a_buf, slot_bytes, base, static_cast<int64_t>(LS) * slot_bytes, 1024) &&
                                   args.a_bytes % 1024 == 0 && (args.r64 & 7) == 0,
                               22)) {
                    // nothing is copied, and the wait for it runs out
                } else if constexpr (!TOK) {
                    tma_load_2d(a_buf, &map_a, bar, k, g.row0);
                    if constexpr (MODE == RANK_T) {
                        tma_load_3d(b_buf, &map_b, bar, k, 0, g.e);
                    } else {
                        for (int c = 0; c < rchunks; ++c) tma_load_3d(b_buf + c * 8192, &map_b, bar, 64 * c, k, g.e);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < kOutRows / 64; ++c)
                        tma_load_2d(a_buf + c * 8192, &map_a, bar, out0 + 64 * c, begin + k);
                    for (int c = 0; c < rchunks; ++c) {
                        tma_load_2d(b_buf + c * 8192, &map_b, bar, 64 * c, begin + k);
                        tma_load_2d(b_buf + (rchunks + c) * 8192, &map_b, bar, args.r64 + 64 * c, begin + k);
                    }
                }
            }
            __syncwarp();
            if (++slot == LS) {
                slot = 0;
                phase ^= 1u;
            }
        }
        if (stop) {
            // let the copies already issued land before the CTA exits
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < 1000000) {}
        }
    } else if (warp == 1) {
        tmem_alloc(&s_tmem, args.tmem_cols);
        tmem_relinquish();
        tc_fence_before();
        asm volatile("bar.arrive 2, %0;" ::"r"(32 + kWork) : "memory");
        __syncwarp();
        tc_fence_after();
        const uint32_t tmem_d = __shfl_sync(0xFFFFFFFFu, s_tmem, 0);
        const uint32_t idesc = make_idesc_bf16(128, 0, TOK ? 1 : 0, MODE == RANK_T ? 0 : 1) |
                               (static_cast<uint32_t>(args.rn >> 3) << 17);
        constexpr uint32_t kAk = TOK ? 2048 / 16 : 32 / 16, kBk = MODE == RANK_T ? 32 / 16 : 2048 / 16;
        const uint64_t a0 = tile_desc(smem_u32(base), TOK, 0);
        const uint64_t b0 = tile_desc(smem_u32(base) + args.a_bytes, MODE != RANK_T, 0);
        int slot = 0, run = 0;
        uint32_t phase = 0, tmem_set = tmem_d;
        for (int it = 0; it < n_steps; ++it) {
            const bool last = own_bar(it);
            bool ok = mbar_wait(last ? &bar_last : &bar_full[slot], last ? 0u : phase, abort_flag);
            if (DROP) ok = ok && mbar_wait(&bar_clear[slot], phase, abort_flag);
            else if (last) ok = ok && mbar_wait(&bar_tail, 0, abort_flag);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            tc_fence_after();
            const uint64_t at = a0 + static_cast<uint32_t>(slot) * (slot_bytes / 16);
            const uint64_t bt = b0 + static_cast<uint32_t>(slot) * (slot_bytes / 16);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const uint32_t first = run * 4 + kk > 0 ? 1u : 0u;
                if constexpr (!TOK) {
                    mma1_elect(tmem_set, at + kk * kAk, bt + kk * kBk, idesc, first);
                } else {
                    const uint64_t hi = bt + kk * kBk, lo = hi + rchunks * (8192 / 16);
#pragma unroll
                    for (int ms = 0; ms < 2; ++ms) {
                        mma1_elect(tmem_d + ms * args.rn, at + ms * (16384 / 16) + kk * kAk, hi, idesc, first);
                        mma1_elect(tmem_d + ms * args.rn, at + ms * (16384 / 16) + kk * kAk, lo, idesc, 1u);
                    }
                }
            }
            mma1_commit_elect(&bar_empty[slot]);
            if (++run == args.run_steps && !TOK) {
                run = 0;
                tmem_set += args.rn;
            }
            if (++slot == LS) {
                slot = 0;
                phase ^= 1u;
            }
        }
        mma1_commit_elect(&bar_accum);
    } else {
        const int ew = warp - 2, wt = threadIdx.x - 64;
        // ------------------------------------------------------------ clearing
        if (DROP || has_tail) {
            KeepGen gen;
            if constexpr (DROP) gen.init(args.drop);
            const int it0 = DROP ? 0 : n_steps - 1;
            int slot = it0 % LS;
            uint32_t phase = (it0 / LS) & 1;
            for (int it = it0; it < n_steps; ++it) {
                const bool last = own_bar(it);
                if (!__all_sync(0xFFFFFFFFu,
                                mbar_wait(last ? &bar_last : &bar_full[slot], last ? 0u : phase, abort_flag)))
                    break;
                uint8_t* a = base + slot * slot_bytes;
                const int k = 64 * (step0 + it);
                if constexpr (DROP) {
                    constexpr int kPieces = kOutRows * 8 / kWork;  // 16-byte pieces per thread
                    // flat index in X, in groups of eight elements, of this thread's
                    // first piece; the pieces of a thread are rows of one chunk
                    // column, drop_cols / 8 groups per row apart
                    const int c = wt & 7, row = wt >> 3;
                    constexpr int kRowStep = kWork / 8;  // rows between a thread's pieces
                    int64_t grp;
                    if constexpr (!TOK)
                        grp = (static_cast<int64_t>(g.row0 + row) * args.drop_cols + k + 8 * c) >> 3;
                    else
                        grp = (static_cast<int64_t>(begin + k + row % 64) * args.drop_cols + out0 + 64 * (row / 64) +
                               8 * c) >> 3;
                    const int gcols = args.drop_cols >> 3;
                    // rows of the tile that are the group's
                    const int rows_kept = has_tail && it == n_steps - 1 ? tail_rows : 64;
#pragma unroll
                    for (int i = 0; i < kPieces; ++i) {
                        int off;
                        uint64_t gi;
                        bool inside = true;
                        if constexpr (!TOK) {
                            const int r = row + i * kRowStep;
                            off = r * 128 + ((c ^ (r & 7)) << 4);
                            gi = static_cast<uint64_t>(grp + static_cast<int64_t>(i * kRowStep) * gcols);
                        } else {
                            // rows run over the chunks: chunk r / 64, row r % 64 of it
                            static_assert(kRowStep == 64 || kRowStep == 32 || !TOK, "rows of a chunk");
                            const int r = row + i * kRowStep, chunk = r / 64, rr = r % 64;
                            off = chunk * 8192 + rr * 128 + ((c ^ (rr & 7)) << 4);
                            gi = static_cast<uint64_t>(grp + 8 * (chunk - row / 64) +
                                                       static_cast<int64_t>(rr - row % 64) * gcols);
                            inside = rr < rows_kept;
                        }
                        uint4* at = reinterpret_cast<uint4*>(a + off);
                        if (!NF4_CHECK(in_smem(at, 16, a, args.a_bytes, 16), 23)) continue;
                        uint4 v = *at;
                        uint32_t m[4];
                        gen.masks(gi, m);
                        v.x &= inside ? m[0] : 0u;
                        v.y &= inside ? m[1] : 0u;
                        v.z &= inside ? m[2] : 0u;
                        v.w &= inside ? m[3] : 0u;
                        *at = v;
                    }
                }
                if (TOK && has_tail && it == n_steps - 1) {
                    // rows behind the group's end: whole 128-byte rows of every chunk;
                    // with dropout the activation's are cleared with the pieces above, by
                    // the threads that hold them, so that nobody waits for another warp
                    // here (one whose wait ran out has left this loop)
                    constexpr int kFirst = DROP ? kOutRows / 64 : 0;
                    uint8_t* b_buf = a + args.a_bytes;
                    const int chunks = kOutRows / 64 + 2 * rchunks - kFirst, per = (64 - tail_rows) * 8;
                    for (int p = wt; p < chunks * per; p += kWork) {
                        const int chunk = kFirst + p / per, rem = p % per;
                        uint8_t* src =
                            chunk < kOutRows / 64 ? a + chunk * 8192 : b_buf + (chunk - kOutRows / 64) * 8192;
                        src += tail_rows * 128 + rem * 16;
                        if (NF4_CHECK(in_smem(src, 16, a, slot_bytes, 16), 23))
                            *reinterpret_cast<uint4*>(src) = make_uint4(0, 0, 0, 0);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(DROP ? &bar_clear[slot] : &bar_tail);
                if (++slot == LS) {
                    slot = 0;
                    phase ^= 1u;
                }
            }
        }
        // ------------------------------------------------------------ epilogue
        asm volatile("bar.sync 2, %0;" ::"r"(32 + kWork) : "memory");
        tc_fence_after();
        const uint32_t tmem_d = s_tmem;
        const int q = warp & 3, half = (ew >> 2) & 1;
        const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(&bar_accum, 0, abort_flag) && !*abort_flag);
        tc_fence_after();
        if (TOK) grid_dependency_wait();
        if (ok && ew < 8) {
            // T, V: the two halves of the warps share the columns; dB, dA: they
            // take one accumulator each
            const bool pairs = !TOK && args.pair != nullptr;
            const int cols = TOK ? args.rn : (pairs ? args.r64 : args.rn) / 2;
            const int cbeg = TOK ? 0 : half * cols;
            const int lrow = q * 32 + lane + (TOK ? half * 128 : 0);
            const int row = TOK ? out0 + lrow : g.row0 + lrow;
            const bool row_ok = row < (TOK ? args.rows : g.row_end);
            const uint32_t at = tmem_d + (static_cast<uint32_t>(q * 32) << 16) + (TOK ? half * args.rn : 0);
            const bool direct = part.parts == 1;
            for (int cc = cbeg; cc < cbeg + cols; cc += 8) {
                __syncwarp();  // the lanes' stores differ; tensor memory is read by the whole warp
                uint32_t v[8];
                if (n_steps > 0 && cc < args.rn) {
                    tmem_ld_32x32b_x8(at + cc, v);
                    tmem_ld_wait();
                    if constexpr (!TOK) {
                        uint32_t set = at + cc;
                        for (int done = args.run_steps; done < n_steps; done += args.run_steps) {
                            uint32_t x[8];
                            set += args.rn;
                            tmem_ld_32x32b_x8(set, x);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(x[j]));
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = 0u;  // a group without rows; columns beyond r
                }
                if (!row_ok) continue;
                if (pairs) {
                    float x[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(v[j]) * args.alpha;
                    store_pair(x, row, cc, args.M, args.r, args.r64, args.pair, args.out32);
                } else if constexpr (!TOK) {
                    float* dst = args.part + blockIdx.z * args.part_slice + static_cast<int64_t>(row) * args.rn + cc;
                    if (!NF4_CHECK(in_span(dst, 32, args.part, gridDim.z * args.part_slice * 4, 16), 24)) continue;
                    *reinterpret_cast<uint4*>(dst) = make_uint4(v[0], v[1], v[2], v[3]);
                    *reinterpret_cast<uint4*>(dst + 4) = make_uint4(v[4], v[5], v[6], v[7]);
                } else if constexpr (MODE == RANK_DB) {
                    if (!direct) {
                        float* dst = args.part + static_cast<int64_t>(part.slot + part.part) * args.part_slice +
                                     static_cast<int64_t>(row) * args.rn + cc;
                        if (!NF4_CHECK(in_span(dst, 32, args.part, args.slots * args.part_slice * 4, 16), 24)) continue;
                        *reinterpret_cast<uint4*>(dst) = make_uint4(v[0], v[1], v[2], v[3]);
                        *reinterpret_cast<uint4*>(dst + 4) = make_uint4(v[4], v[5], v[6], v[7]);
                    } else {
                        uint16_t* dst = args.out + (static_cast<int64_t>(g.e) * args.rows + row) * args.r + cc;
                        if (cc >= args.r) continue;
                        if (!NF4_CHECK(in_span(dst, 2 * min(8, args.r - cc), args.out,
                                               static_cast<int64_t>(args.E) * args.rows * args.r * 2,
                                               args.r % 8 == 0 ? 16 : 2),
                                       25))
                            continue;
                        uint16_t o[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            float x = __uint_as_float(v[j]) * args.alpha;
                            if (args.accumulate && cc + j < args.r) x += bf16_bits_to_float(dst[j]);
                            o[j] = bf16_bits(x);
                        }
                        if (args.r % 8 == 0) {
                            if (cc < args.r) *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(o);
                        } else {
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                if (cc + j < args.r) dst[j] = o[j];
                        }
                    }
                } else {
                    if (!direct) {
                        float* dst = args.part + static_cast<int64_t>(part.slot + part.part) * args.part_slice +
                                     static_cast<int64_t>(cc) * args.rows + row;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (NF4_CHECK(in_span(dst + static_cast<int64_t>(j) * args.rows, 4, args.part,
                                                  args.slots * args.part_slice * 4, 4),
                                          24))
                                dst[static_cast<int64_t>(j) * args.rows] = __uint_as_float(v[j]);
                    } else {
                        uint16_t* dst = args.out + (static_cast<int64_t>(g.e) * args.r + cc) * args.rows + row;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (cc + j < args.r) {
                                uint16_t* d = dst + static_cast<int64_t>(j) * args.rows;
                                if (!NF4_CHECK(in_span(d, 2, args.out,
                                                       static_cast<int64_t>(args.E) * args.rows * args.r * 2, 2),
                                               25))
                                    continue;
                                float x = __uint_as_float(v[j]) * args.alpha;
                                if (args.accumulate) x += bf16_bits_to_float(*d);
                                *d = bf16_bits(x);
                            }
                    }
                }
            }
        }
    }
    __syncwarp();
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
};

__global__ void k_rank_rows_sum(const RankRowsSumArgs a) {
    grid_dependency_wait();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int lo = 0, hi = a.M;
    if (a.offsets != nullptr) {
        lo = min(max(__ldcg(a.offsets), 0), a.M);
        hi = min(max(__ldcg(a.offsets + a.E), lo), a.M);
    }
    const int octs = a.r64 / 8;
    const int64_t total = static_cast<int64_t>(hi - lo) * octs;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t row = lo + i / octs;
        const int j = 8 * static_cast<int>(i % octs);
        float v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = 0.0f;
        if (j < a.rn) {
            const float* p = a.part + row * a.rn + j;
            for (int z = 0; z < a.splits; ++z, p += a.slice) {
                if (!NF4_CHECK(in_span(p, 32, a.part, a.splits * a.slice * 4, 16), 26)) break;
                const float4 x = __ldcg(reinterpret_cast<const float4*>(p));
                const float4 y = __ldcg(reinterpret_cast<const float4*>(p) + 1);
                v[0] += x.x;
                v[1] += x.y;
                v[2] += x.z;
                v[3] += x.w;
                v[4] += y.x;
                v[5] += y.y;
                v[6] += y.z;
                v[7] += y.w;
            }
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] *= a.alpha;
        store_pair(v, row, j, a.M, a.r, a.r64, a.pair, a.out32);
    }
}

// The pair of a saved fp32 T [M, r].
__global__ void k_rank_pair(const float* __restrict__ src, int64_t M, int r, int r64, uint16_t* __restrict__ pair) {
    grid_dependency_wait();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int octs = r64 / 8;
    const int64_t total = M * octs;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t row = i / octs;
        const int j = 8 * static_cast<int>(i % octs);
        float v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = j + u < r ? __ldcg(src + row * r + j + u) : 0.0f;
        store_pair(v, row, j, M, r, r64, pair, nullptr);
    }
}

// dB [E][N][r] (TRANSPOSED false) or dA [E][r][K] of the groups of several parts,
// from partials [part][N][rn] or [part][rn][K], added in order.  Each block lists
// those groups first and takes its share of their elements, so that the many
// groups of one part cost nothing (a block per expert: 18 and 23 us for 64 experts
// of 2048 x 1408, of which a few have several parts).  The list has room for `cap`
// groups, which is min(E, slots / 2) and so all that valid offsets can make; it
// lies in dynamic shared memory so that blocks fit beside the next kernel's.  VEC
// elements at a time (4 needs r to be a multiple of 4 where not TRANSPOSED).
constexpr int kSumGroupBytes = 10;
template <bool TRANSPOSED, int VEC>
__global__ void __launch_bounds__(256)
    k_rank_grad_sum(const int32_t* offsets, int E, int M, int part_steps, int slots, const float* __restrict__ part,
                    int rows, int r, int rn, float alpha, uint16_t* __restrict__ out, int accumulate, int cap) {
    extern __shared__ int s_list[];
    int *s_slot = s_list, *s_parts = s_list + cap;
    uint16_t* s_e = reinterpret_cast<uint16_t*>(s_list + 2 * cap);
    __shared__ int s_warp[8][2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // the offsets were complete before the kernels that this one follows
    int groups = 0, slot0 = 0;
    for (int e0 = 0; e0 < E; e0 += 256) {
        const int e = e0 + threadIdx.x;
        int begin = 0, end = 0;
        if (e < E) {
            if (offsets != nullptr) group_bounds(offsets, e, M, begin, end);
            else end = M;
        }
        const int n = rank_parts(end - begin, part_steps), taken = n > 1 ? n : 0;
        int g = n > 1 ? 1 : 0, sl = taken;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, g, d), w = __shfl_up_sync(0xFFFFFFFFu, sl, d);
            if (lane >= d) {
                g += v;
                sl += w;
            }
        }
        if (lane == 31) {
            s_warp[warp][0] = g;
            s_warp[warp][1] = sl;
        }
        __syncthreads();
        int g_all = 0, sl_all = 0;
        for (int w = 0; w < 8; ++w) {
            if (w == warp) {
                g += g_all;
                sl += sl_all;
            }
            g_all += s_warp[w][0];
            sl_all += s_warp[w][1];
        }
        const int k = groups + g - 1;
        if (n > 1 && k < cap) {
            s_e[k] = static_cast<uint16_t>(e);
            s_slot[k] = slot0 + sl - taken;
            // what the slots do not hold was written as one part (offsets that
            // break their contract)
            s_parts[k] = slot0 + sl <= slots ? n : 0;
        }
        groups += g_all;
        slot0 += sl_all;
        __syncthreads();
    }
    groups = min(groups, cap);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    grid_dependency_wait();
    const int64_t slice = static_cast<int64_t>(rows) * rn;
    const int inner = (TRANSPOSED ? rows : r) / VEC, ld = TRANSPOSED ? rows : rn;
    const int64_t total = static_cast<int64_t>(rows) * r / VEC, chunks = (total + 255) / 256;
    for (int64_t u = blockIdx.x; u < groups * chunks; u += gridDim.x) {
        const int k = static_cast<int>(u / chunks), parts = s_parts[k];
        const int64_t i = (u - k * chunks) * 256 + threadIdx.x;
        if (parts == 0 || i >= total) continue;
        uint16_t* dst = out + static_cast<int64_t>(s_e[k]) * rows * r;
        const int64_t outer = total < (int64_t(1) << 31) ? static_cast<int>(i) / inner : i / inner;
        const float* at = part + s_slot[k] * slice + outer * ld + (i - outer * inner) * VEC;
        if (!NF4_CHECK(in_span(at, 4 * VEC, part, slots * slice * 4, 4 * VEC) &&
                           in_span(at + (parts - 1) * slice, 4 * VEC, part, slots * slice * 4, 4 * VEC) &&
                           in_span(dst + i * VEC, 2 * VEC, out, static_cast<int64_t>(E) * rows * r * 2, 2 * VEC),
                       27))
            continue;
        float v[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] = 0.0f;
#pragma unroll 4
        for (int z = 0; z < parts; ++z) {
            if constexpr (VEC == 4) {
                const float4 x = __ldcg(reinterpret_cast<const float4*>(at + z * slice));
                v[0] += x.x;
                v[1] += x.y;
                v[2] += x.z;
                v[3] += x.w;
            } else {
                v[0] += __ldcg(at + z * slice);
            }
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            v[j] *= alpha;
            if (accumulate) v[j] += bf16_bits_to_float(dst[i * VEC + j]);
        }
        if constexpr (VEC == 4)
            reinterpret_cast<uint2*>(dst)[i] = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        else
            dst[i] = bf16_bits(v[0]);
    }
}

}  // namespace nf4lora
