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
// The pairs are persistent: pair i takes the tiles i, i + pairs, ... and keeps
// its barriers, rings and tensor memory; the copies and decodes of the next tile
// run while the epilogue of the last one empties the accumulators.  The groups'
// bounds are device data: a CTA lists them once (up to 127 groups; beyond, each
// warp finds its tiles by scans of the offsets), and the first tile beyond the
// last group ends the walk.  A group of n rows is divided evenly into tiles of at
// most tile_rows.  A tile never crosses a group: rows of the
// next group that its copies bring in are accumulator columns that are not
// stored, or beyond N altogether.  With few tokens the contraction is split too
// (fp32 partials, added in order by k_group_sum), so that the tiles divide evenly
// over the pairs.
//
// Weights and factors are three-dimensional tensor maps (inner, row, expert):
// rows beyond an expert's own read as zeros and never as the next expert's, so
// a NaN or an infinity in one expert's adapter cannot reach another's result.
//
// Warp roles, in each CTA: warp 0 copies (TMA); warp 1 owns tensor memory and in
// the leading CTA issues the MMAs; teams of four or eight warps decode k-steps in
// turn and run the epilogue; with one CTA per SM a last warp copies the packed
// codes.  Rings: steps (tokens and decoded tiles) and packed codes.  One barrier
// of the leading CTA collects, for a step, the bytes of both CTAs' tokens and both
// teams' arrivals: the issuing warp waits once a step, and polls the next step's
// barrier beside the MMAs.  The rank-r term enters the same accumulator as
// extension k-steps over [hi | lo] of the 16-bit pair of T or V.
//
// What bounds it (B200, CUDA graph, whole calls): many tokens, the tensor pipe
// (4096 tokens, 4096 -> 11008: 249 us, 1480 TFLOP/s); a couple of hundred tokens a
// group, the decode, 850 clocks a 64-deep step of which the integer or the
// shared-memory pipe needs 300 to 500 and latencies of the decoding warps the
// rest; few tokens, the decode too (64 tokens over eight experts of 4096 x 11008:
// 105 us for 186 MB of codes and scales).
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

__device__ __forceinline__ void tmem_st_32x32b_x8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

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
    int row_end;  // end of its rows (EVEN tiles) or of the group's
};

// Bounds of group e, clamped into 0 <= begin <= end <= M, so that offsets that
// break the contract can never lead an access out of the arrays.
__device__ __forceinline__ void group_bounds(const int32_t* offsets, int e, int M, int& begin, int& end) {
    begin = min(max(__ldcg(offsets + e), 0), M);
    end = min(max(__ldcg(offsets + e + 1), begin), M);
}

// Tile t of all groups' tiles of at most `most` rows, in group order; the whole
// warp calls it.  EVEN: a group's tiles are of one size, a multiple of 32, else
// all but its last have `most` rows.  bounds(e, begin, end) gives a group's rows.
// False beyond the last tile.
template <bool EVEN, typename Bounds>
__device__ __forceinline__ bool find_tile(bool grouped, const Bounds& bounds, int E, int M, int most, int t, int lane,
                                          GroupTile& g) {
    int begin = 0, end = M, first = 0;
    g.e = 0;
    if (grouped) {
        bool found = false;
        for (int e0 = 0; e0 < E && !found; e0 += 32) {
            const int e = e0 + lane;
            begin = end = 0;
            if (e < E) bounds(e, begin, end);
            const int n = (end - begin + most - 1) / most;
            int incl = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
                if (lane >= d) incl += v;
            }
            const unsigned hit = __ballot_sync(0xFFFFFFFFu, first + incl > t);
            if (hit != 0) {
                const int src = __ffs(hit) - 1;
                g.e = e0 + src;
                first += __shfl_sync(0xFFFFFFFFu, incl - n, src);
                begin = __shfl_sync(0xFFFFFFFFu, begin, src);
                end = __shfl_sync(0xFFFFFFFFu, end, src);
                found = true;
            } else {
                first += __shfl_sync(0xFFFFFFFFu, incl, 31);
            }
        }
        if (!found) return false;
    }
    int size = most;
    if (EVEN) {
        const int n = end - begin, k = (n + most - 1) / most;
        size = k > 0 ? ((n + k - 1) / k + 31) & ~31 : most;
    }
    g.row0 = begin + (t - first) * size;
    g.row_end = EVEN ? min(end, g.row0 + size) : end;
    return g.row0 < end;
}

// The same with the bounds from device memory.
template <bool EVEN>
__device__ __forceinline__ bool find_tile(const int32_t* offsets, int E, int M, int most, int t, int lane,
                                          GroupTile& g) {
    auto bounds = [&](int e, int& begin, int& end) { group_bounds(offsets, e, M, begin, end); };
    return find_tile<EVEN>(offsets != nullptr, bounds, E, M, most, t, lane, g);
}

// ------------------------------------------------------------------ one thread of a warp
// The MMA and copy instructions take their operands from uniform registers.
// They are issued from code that the whole (converged) warp runs on uniform
// values, by the one thread that elect.sync names; under a condition on the lane
// index the compiler has to assume that values differ between threads and wraps
// every such instruction in a loop over them (measured: about 120 clocks an MMA).
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(e));
    return e != 0;
}

__device__ __forceinline__ void mma1_elect(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "elect.sync _|e, 0xFFFFFFFF;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrive once on `bar` when every MMA issued so far has completed.
__device__ __forceinline__ void mma1_commit_elect(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xFFFFFFFF;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}

// ------------------------------------------------------------------ CTA pairs
__device__ __forceinline__ void mma2_elect(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "elect.sync _|e, 0xFFFFFFFF;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Whether the phase is complete, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Four of them, 64 deep, issued by one elected lane; kA and kB: from one 16 of the
// contraction to the next, in descriptor units.
template <int kA, int kB>
__device__ __forceinline__ void mma2_elect4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, t, e;\n\t.reg .b64 a, b;\n\t"
        "elect.sync _|e, 0xFFFFFFFF;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.eq.b32 t, 0, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "add.s64 a, %1, %5;\n\tadd.s64 b, %2, %6;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, t;\n\t"
        "add.s64 a, %1, 2 * %5;\n\tadd.s64 b, %2, 2 * %6;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, t;\n\t"
        "add.s64 a, %1, 3 * %5;\n\tadd.s64 b, %2, 3 * %6;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, t;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "n"(kA), "n"(kB)
        : "memory");
}

// The same with operand A in tensor memory: 128 lanes (rows) of each CTA by 8
// columns, two bf16 of the contraction in a column.
__device__ __forceinline__ void mma2_elect_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "elect.sync _|e, 0xFFFFFFFF;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrive once on `bar` of both CTAs of the pair when every MMA issued so far
// has completed.
__device__ __forceinline__ void mma2_commit_elect(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xFFFFFFFF;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

// A copy into this CTA's shared memory that completes on a barrier of either CTA
// of the pair (a shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(void* smem_dst, const CUtensorMap* map, uint32_t cluster_bar,
                                                 int32_t x, int32_t y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(cluster_bar), "r"(x), "r"(y)
        : "memory");
}

__device__ __forceinline__ void tma_load_3d_pair(void* smem_dst, const CUtensorMap* map, uint32_t cluster_bar,
                                                 int32_t x, int32_t y, int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(cluster_bar), "r"(x), "r"(y), "r"(z)
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

// ------------------------------------------------------------------ decode
// One (weight row, 64-block) unit: 32 packed bytes to 64 bf16.  Two look-ups:
//
// decode_word, eight codes by byte permutes: that of csrc/decode.cuh with the
// selectors formed for a whole code word; the permutes and logic run on the
// integer pipe at half rate and bound it, so the shifts are written as high
// halves of products, which run on the multiply pipe.  370 clocks per SM for the
// units of four warps.
//
// shuffle_word: each level comes from the lane that holds it (`level`: of this
// lane's index modulo 16), and the products are rounded as they come, which needs
// no table and no logic but takes the shared-memory pipe: 252 clocks (look-ups in
// shared memory: 293; mixtures of the two: in between).
__device__ __forceinline__ void decode_word(uint32_t w, const uint32_t (&P)[4], const uint32_t (&H)[4], uint32_t* o) {
    const uint32_t sel = w & 0x77777777u;                                          // index within 0-7 / 8-15
    const uint32_t pick = (__umulhi(w, 0x80000000u) & 0x44444444u) | 0x32103210u;  // from 8-15 if bit 3
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t se = h ? __umulhi(sel, 0x10000u) : sel, pk = h ? __umulhi(pick, 0x10000u) : pick;
        const uint32_t lo = __byte_perm(__byte_perm(P[0], P[1], se), __byte_perm(P[2], P[3], se), pk);
        const uint32_t hi = __byte_perm(__byte_perm(H[0], H[1], se), __byte_perm(H[2], H[3], se), pk);
        o[2 * h] = __byte_perm(lo, hi, 0x4051);
        o[2 * h + 1] = __byte_perm(lo, hi, 0x6273);
    }
}

__device__ __forceinline__ void shuffle_word(uint32_t w, float s, float level, uint32_t* o) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float even = __shfl_sync(0xFFFFFFFFu, level, w >> (8 * i + 4), 16);
        const float odd = __shfl_sync(0xFFFFFFFFu, level, w >> 8 * i, 16);
        o[i] = pack_bf16x2(__fmul_rn(even, s), __fmul_rn(odd, s));
    }
}

// A unit as the 8 swizzled 16-byte chunks of one 128-byte row (dst: the row's
// address with the swizzle's XOR already in it); the whole warp calls it.  Tiles
// of up to 256 tokens take the shuffles (125 tokens in each of 64 experts of
// 2048 x 1408, a training step: 295 us against 301), the larger ones, whose MMAs
// and copies need the shared-memory pipe, the permutes (188 tokens in each of
// eight of 4096 x 11008: 390 against 402).
template <bool SHUFFLE>
__device__ __forceinline__ void decode_row(const uint8_t* src, float s, float level, uint8_t* dst) {
    uint32_t P[4], H[4];
    if constexpr (!SHUFFLE) nf4_table(s, P, H);
    const uint4 c0 = *reinterpret_cast<const uint4*>(src);
    const uint4 c1 = *reinterpret_cast<const uint4*>(src + 16);
    const uint32_t words[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
    const uint32_t at = smem_u32(dst);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        uint32_t o[4];
        if constexpr (SHUFFLE) shuffle_word(words[j], s, level, o);
        else decode_word(words[j], P, H, o);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at ^ (j << 4)), "r"(o[0]), "r"(o[1]), "r"(o[2]),
                     "r"(o[3])
                     : "memory");
    }
}

// A unit in tensor memory: 32 columns of the thread's lane from `taddr` on (the
// warp's lane base in it), two weights a column; the whole warp calls it, and
// waits for the stores itself.
__device__ __forceinline__ void decode_lane(const uint8_t* src, float s, float level, uint32_t taddr) {
    const uint4 c0 = *reinterpret_cast<const uint4*>(src);
    const uint4 c1 = *reinterpret_cast<const uint4*>(src + 16);
    const uint32_t words[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        uint32_t o[8];
        shuffle_word(words[j], s, level, o);
        shuffle_word(words[j + 1], s, level, o + 4);
        tmem_st_32x32b_x8(taddr + 4 * j, o);
    }
}

// ------------------------------------------------------------------ fused product
struct GroupGemmArgs {
    const int32_t* offsets;  // [E + 1], or NULL
    int E;
    int M;
    int cols;                // forward: N; input gradient: K
    int k_main;              // steps of the contraction (64 kKS wide)
    int k_ext;               // extension steps over 2 r64 (split 0)
    int splits;              // parts of the contraction; > 1: partials
    int tile_rows;           // at most, a multiple of 32
    int col_tiles;
    int row_tiles;           // walked first when >= 0 (one dense group, its exact count), else the column tiles are
    int most_row_tiles;      // that any division of the rows can need
    int walk_z, walk_fast, walk_slow;  // number of pairs = walk_z + splits (walk_fast + fast tiles walk_slow)
    // encoded weight: rows and blocks of one expert
    const int8_t* qscale;
    const float* scale2;
    const float* scale_mean;
    const float* absmax;
    int w_rows;
    int w_blocks_per_row;
    uint16_t* out;           // [M, cols]
    float* part;             // [splits][M][cols]
    DropArgs drop;           // input gradient with dropout only
};

// Tensor maps of the same rows with boxes of kBoxRows, 2 kBoxRows, ...: a tile's
// copies bring the rows it has and not the largest tile's.
struct RowMaps {
    CUtensorMap m[4];
};

// T tokens per tile at most.
//
// 512: one CTA per SM, four teams, steps of 64, one set of accumulators; the MMAs,
// and with fewer than 350 tokens their issue, bound it.
//
// 256: the decode bounds it; steps of 128 by teams of eight warps (half the waits,
// arrivals and turns of the copying and issuing warps per decoded weight).  Input
// gradient: two sets of accumulators, so that MMAs run beside the epilogue; forward:
// one, and the decoded tiles beside it in tensor memory (kWT, as below; 188 tokens
// in each of eight experts of 4096 x 11008, a training step: 362 us against 384).
//
// 64 (forward), 32 (input gradient): two CTAs per SM of two teams each, whose
// starts and ends overlap, and steps of 128 (two units per thread; steps of 64:
// 167 us for 64 tokens over eight experts of 4096 x 11008, steps of 128: 143 us).
// Forward (kWT): the tile is K-major, lane = weight row, and goes to tensor memory
// (32 columns a unit; three steps fit beside the accumulators), by which the
// shared-memory pipe is free to do the look-ups as shuffles: 105 us.  Input
// gradient: the tile is MN-major, which only shared memory can hold, two steps of
// it; with 64 tokens those would be 242 us against 217 (a step of 16 tokens in each
// of 64 experts of 2048 x 1408).
template <bool DX, int T>
struct GroupGemmConfig {
    static constexpr int kBM = 128;                    // weight columns of one CTA
    static constexpr int kSubs = T > 256 ? 2 : 1;      // accumulators
    static constexpr int kSubT = T / kSubs;            // tokens of one, half of them per CTA
    static constexpr bool kWT = T <= 256 && !DX;  // decoded weights in tensor memory
    static constexpr int kTeams = T > 256 ? 4 : 2;
    static constexpr int kKS = T > 256 ? 1 : 2;        // 64s of the contraction in a step
    static constexpr int kUnits = T > 64 ? 1 : 2;      // (row, block) units of a step per thread
    static constexpr int kDS = T > 256 || (T > 64 && kWT) ? 4 : T > 64 || kWT ? 3 : 2;  // slots of steps
    static constexpr int kLC = T > 256 ? 8 : T > 64 ? 4 : 2 * kDS;   // slots of packed codes
    static constexpr int kWS = kWT ? 1 : kDS;          // slots of weight tiles in shared memory (kWT: extension only)
    static constexpr int kBoxRows = T > 64 ? 32 : 16, kBoxes = kSubT / 2 / kBoxRows;
    static constexpr int kSub = kSubT / 2 * 128;       // a CTA's tokens of one accumulator, 64 deep
    static constexpr int kTok = kSubs * kSub;          // of all accumulators
    static constexpr int kCodes = kBM * 32, kW = kBM * 128;  // a packed and a decoded tile, 64 deep
    static constexpr int kTokBytes = kKS * kTok, kCBytes = kKS * kCodes, kWBytes = kKS * kW;
    static constexpr int kSmem = kDS * kTokBytes + kWS * kWBytes + kLC * kCBytes + 1024;
    static constexpr int kTeamThreads = kBM * (kKS / kUnits);
    static constexpr int kTeamWarps = kTeamThreads / 32;
    static constexpr int kWorkWarps = kTeamWarps * kTeams;
    // With one CTA per SM a warp of its own copies the codes, into slots that the
    // decoders free (else the copying warp's turns, some 600 clocks a step, bound
    // all tiles of few tokens); with two the registers do not go round for it.
    static constexpr bool kCodeWarp = T > 64;
    static constexpr int kThreads = 64 + 32 * kWorkWarps + (kCodeWarp ? 32 : 0);
    static constexpr int kMinBlocks = T > 64 ? 1 : 2;
    static constexpr int kAccs = T > 256 || kWT ? 1 : 2;  // sets of accumulators; two: MMAs run beside the epilogue
    static constexpr int kAccCols = T;                 // columns of a set
    static constexpr int kTmemCols = kWT ? (T > 64 ? 512 : 256) : kAccs * T;
    static constexpr uint32_t kIdesc = make_idesc_bf16(2 * kBM, 0, DX ? 1 : 0, 0);  // without N
    // A wait for a barrier's phase is sound only where the phase before it is
    // known to be complete.  Code slots: a slot is always the same team's.  Decode
    // slots: that phase is of the step 2 kDS before, not after the one whose MMAs
    // (they complete in order) the team has waited for at its last step.
    static_assert(kDS >= kTeams && kLC % kTeams == 0 && kLC >= kDS, "rings");
    static_assert(!kWT || kAccs * T + kDS * kKS * 32 <= kTmemCols, "tensor memory");
    static_assert(kSub % 1024 == 0 && kSmem * kMinBlocks <= 226 * 1024, "shared memory");
};

// map_t: X [M, K] or dY [M, N], boxes {64, kBoxRows ...}.  map_w: codes (K / 2, N,
// E), box {32, 128, 1} (forward) or {64, 64, 1}.  map_te: T2 or V2 [M, 2 r64],
// boxes as map_t's.  map_we: B (r, N, E), box {64, 128, 1} (forward) or A (K,
// r, E), box {64, 64, 1}.  Cluster of two along grid.x.
template <bool DX, int T, bool DROP>
__global__ void __launch_bounds__(GroupGemmConfig<DX, T>::kThreads, GroupGemmConfig<DX, T>::kMinBlocks)
    k_group_gemm(const __grid_constant__ RowMaps map_t, const __grid_constant__ CUtensorMap map_w,
                 const __grid_constant__ RowMaps map_te, const __grid_constant__ CUtensorMap map_we,
                 const GroupGemmArgs args) {
    using C = GroupGemmConfig<DX, T>;
    static_assert(DX || !DROP, "only the input gradient masks its accumulator");
    constexpr int LC = C::kLC, DS = C::kDS;
    constexpr int kWork = C::kWorkWarps * 32;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    // bar_ready, bar_masked and bar_free count both CTAs, in the leading one
    // (rank 0); the MMAs' completions (bar_done, bar_accum, bar_ext) arrive in
    // both; bar_codes and bar_cfree are each CTA's own
    __shared__ uint64_t bar_codes[LC], bar_cfree[LC], bar_ready[DS], bar_done[DS], bar_accum[C::kAccs], bar_ext,
        bar_masked, bar_free[C::kAccs];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    // The groups' rows, first tiles and tile sizes, worked out once; for more
    // groups than this a warp scans the offsets for every tile.
    constexpr int kGroups = 127;
    __shared__ int s_off[kGroups + 1], s_first[kGroups + 1];
    __shared__ uint16_t s_size[kGroups + 1];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    // the offsets, the activations and the encoded weight were complete before
    // the kernel this one depends on released it (that kernel waited for all
    // earlier ones first); T2 / V2 is that kernel's and is waited for below, after
    // which this one releases its own dependents

    // A tile of this pair.  Its steps: n_main of the contraction from kb0 on, and
    // in the first split the n_ext extension steps -- after them, or with dropout
    // before.
    struct Tile {
        GroupTile g;
        int h0;      // weight columns of this CTA
        int tokens;
        int nsub;
        int z, kb0, n_main, n_ext;
    };
    const bool kept = args.offsets != nullptr && args.E <= kGroups;
    // The walk over this pair's tiles: tile i = pair + tl pairs is split z of
    // column tile ct and token tile rt, kept as running numbers (the steps of a
    // walk, pairs = dct + col_tiles (drt + ...), come from the host: a division
    // costs as much as a good part of a decode).
    struct Walk {
        int z, fast, slow;
    };
    const int fast_n = args.row_tiles >= 0 ? args.row_tiles : args.col_tiles;
    auto first_tile = [&](Walk& w) {
        const int i = blockIdx.x >> 1;
        w.z = i % args.splits;
        w.fast = i / args.splits % fast_n;
        w.slow = i / args.splits / fast_n;
    };
    auto next_tile = [&](Walk& w, Tile& t) {
        t.z = w.z;
        const int ct = args.row_tiles >= 0 ? w.slow : w.fast, rt = args.row_tiles >= 0 ? w.fast : w.slow;
        w.z += args.walk_z;
        w.fast += args.walk_fast;
        w.slow += args.walk_slow;
        if (w.z >= args.splits) {
            w.z -= args.splits;
            ++w.fast;
        }
        if (w.fast >= fast_n) {
            w.fast -= fast_n;
            ++w.slow;
        }
        // offsets that break their rule may ask for more tiles than the rows can have
        // (every group may be clamped to all rows): those are left out
        if (ct >= args.col_tiles || rt >= args.most_row_tiles) return false;
        if (kept) {
            // the last group whose first tile is not beyond rt (groups without rows
            // share their first tile with the next one)
            int e = -1;
            for (int e0 = 0; e0 < args.E; e0 += 32)
                e += __popc(__ballot_sync(0xFFFFFFFFu, e0 + lane < args.E && s_first[min(e0 + lane, kGroups)] <= rt));
            if (rt >= s_first[args.E]) return false;
            if (!NF4_CHECK(e >= 0 && e < args.E, 32)) return false;
            const int begin = min(max(s_off[e], 0), args.M);
            t.g.e = e;
            t.g.row0 = begin + (rt - s_first[e]) * s_size[e];
            t.g.row_end = min(min(max(s_off[e + 1], begin), args.M), t.g.row0 + s_size[e]);
        } else if (!find_tile<true>(args.offsets, args.E, args.M, args.tile_rows, rt, lane, t.g)) {
            return false;
        }
        t.h0 = (2 * ct + rank) * C::kBM;
        t.tokens = t.g.row_end - t.g.row0;
        t.nsub = C::kSubs == 2 && t.tokens > C::kSubT ? 2 : 1;
        t.kb0 = 0;
        t.n_main = args.k_main;
        if (args.splits > 1) {
            t.kb0 = args.k_main * t.z / args.splits;
            t.n_main = args.k_main * (t.z + 1) / args.splits - t.kb0;
        }
        t.n_ext = t.z == 0 ? args.k_ext : 0;
        return true;
    };
    // N of accumulator s, and the first of the rows that this CTA brings for it
    auto sub_n = [&](const Tile& t, int s) { return (min(C::kSubT, t.tokens - s * C::kSubT) + 31) & ~31; };
    auto sub_row = [&](const Tile& t, int s) { return t.g.row0 + s * C::kSubT + rank * (sub_n(t, s) >> 1); };
    auto main0 = [&](const Tile& t) { return DROP ? t.n_ext : 0; };
    auto is_main = [&](const Tile& t, int it) { return DROP ? it >= t.n_ext : it < t.n_main; };

    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* base = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    // Buffers: a step's slot ds, code slot cs, and its weight slot: ds, or with the
    // decoded tiles in tensor memory the extension steps' own one
    auto t_buf = [&](int ds) { return base + ds * C::kTokBytes; };
    auto w_buf = [&](int ws) { return base + DS * C::kTokBytes + ws * C::kWBytes; };
    auto codes_buf = [&](int cs) { return base + DS * C::kTokBytes + C::kWS * C::kWBytes + cs * C::kCBytes; };

    if (threadIdx.x == 0) {
        for (int i = 0; i < LC; ++i) {
            mbar_init(&bar_codes[i], 1);
            mbar_init(&bar_cfree[i], C::kTeamWarps);
        }
        for (int i = 0; i < DS; ++i) {
            mbar_init(&bar_ready[i], 1 + 2 * C::kTeamWarps);
            mbar_init(&bar_done[i], 1);
        }
        for (int i = 0; i < C::kAccs; ++i) {
            mbar_init(&bar_accum[i], 1);
            mbar_init(&bar_free[i], 2 * C::kWorkWarps);
        }
        mbar_init(&bar_ext, 1);
        mbar_init(&bar_masked, 2 * C::kWorkWarps);
        s_abort = 0;
        fence_barrier_init();
    }
    if (kept && warp == 1) {
        int tiles = 0;
        for (int e0 = 0; e0 <= args.E; e0 += 32) {
            const int e = e0 + lane;
            int begin = 0, end = 0;
            if (e < args.E) group_bounds(args.offsets, e, args.M, begin, end);
            const int n = end - begin, k = (n + args.tile_rows - 1) / args.tile_rows;
            int incl = k;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
                if (lane >= d) incl += v;
            }
            if (e <= args.E) {
                s_off[e] = __ldcg(args.offsets + e);
                s_first[e] = tiles + incl - k;
                s_size[e] = static_cast<uint16_t>(k > 0 ? ((n + k - 1) / k + 31) & ~31 : 0);
            }
            tiles = min(tiles + __shfl_sync(0xFFFFFFFFu, incl, 31), args.most_row_tiles);
        }
    }
    // both CTAs' barriers are initialised once this barrier is passed
    cluster_arrive_release();
    cluster_wait_acquire();
    volatile int* abort_flag = &s_abort;
    // the leading CTA's copy of a barrier (shared::cluster address)
    auto lead = [&](uint64_t* bar) { return cluster_map(smem_u32(bar), 0); };

    // packed codes of step it into slot cs; an extension step, whose factor tile
    // goes with its tokens, completes the slot's phase without any.  The whole warp
    // calls it.
    auto load_codes = [&](const Tile& t, int it, int cs) {
        if (elect_one() && NF4_CHECK(cs < LC && in_smem(codes_buf(cs), C::kCBytes, base, C::kSmem - 1024, 1024), 30)) {
            uint64_t* bar = &bar_codes[cs];
            if (is_main(t, it)) {
                mbar_arrive_expect_tx(bar, C::kCBytes);
                const int kb = (t.kb0 + it - main0(t)) * C::kKS;
#pragma unroll
                for (int h = 0; h < C::kKS; ++h) {
                    uint8_t* dst = codes_buf(cs) + h * C::kCodes;
                    if constexpr (DX) tma_load_3d(dst, &map_w, bar, t.h0 / 2, (kb + h) * 64, t.g.e);
                    else tma_load_3d(dst, &map_w, bar, (kb + h) * 32, t.h0, t.g.e);
                }
            } else {
                mbar_arrive(bar);
            }
        }
        __syncwarp();
    };

    if (warp == 0) {
        // ------------------------------------------------------------ copies
        if (lane == 0) {
            tma_prefetch_desc(&map_w);
            tma_prefetch_desc(&map_we);
        }
        __syncwarp();
        bool waited = false;
        // without a warp of their own the codes run kAhead steps before the tokens,
        // into the next tile
        constexpr int kAhead = C::kCodeWarp ? 0 : LC - DS;
        Tile tc, tt;  // tiles of the codes' and of the tokens' step
        Walk wc, wt;
        first_tile(wc);
        wt = wc;
        int itc = 0, csc = 0;
        bool have_c = !C::kCodeWarp && next_tile(wc, tc);
        auto codes_step = [&]() {
            if (C::kCodeWarp || !have_c) return;
            load_codes(tc, itc, csc);
            if (++csc == LC) csc = 0;
            if (++itc == tc.n_main + tc.n_ext) {
                itc = 0;
                have_c = next_tile(wc, tc);
            }
        };
        for (int i = 0; i < kAhead; ++i) codes_step();
        int ds = 0;             // slot of the tokens' step
        uint32_t done = 0;      // parity of the round over the slots
        int since = DS;         // steps since the last extension step (kWT)
        bool stop = false;
        while (!stop && next_tile(wt, tt)) {
            const int n_iter = tt.n_main + tt.n_ext;
            // the boxes that hold the rows this CTA brings for an accumulator
            int box[C::kSubs], bytes = 0;
#pragma unroll
            for (int ms = 0; ms < C::kSubs; ++ms) {
                box[ms] = min(max(0, ((sub_n(tt, ms) >> 1) - 1) / C::kBoxRows), C::kBoxes - 1);
                if (ms < tt.nsub) bytes += C::kKS * (box[ms] + 1) * C::kBoxRows * 128;
            }
            for (int it = 0; it < n_iter; ++it) {
                // the step DS before is multiplied: its token and decode slots are
                // free, and so is the code slot of the step kAhead ahead, which its
                // decode has read.  The warp stays together also when a wait gives up.
                stop = __any_sync(0xFFFFFFFFu, !mbar_wait(&bar_done[ds], done ^ 1u, abort_flag) || *abort_flag);
                if (stop) break;
                const bool main_step = is_main(tt, it);
                const int j0 = (DROP ? it : it - tt.n_main) * C::kKS;  // of an extension step
                if (C::kWT && !main_step) {
                    // the one slot of factors: free once the last extension step is
                    // multiplied (DS or more steps back it is known to be)
                    if (since < DS) {
                        const int back = ds >= since ? ds - since : ds - since + DS;
                        const uint32_t parity = ds >= since ? done : done ^ 1u;
                        stop = __any_sync(0xFFFFFFFFu, !mbar_wait(&bar_done[back], parity, abort_flag));
                        if (stop) break;
                    }
                    since = 0;
                }
                if (C::kWT) since = min(since + 1, DS);
                if (elect_one() &&
                    NF4_CHECK(ds < DS && in_smem(t_buf(ds), C::kTokBytes, base, C::kSmem - 1024, 1024) &&
                                  in_smem(w_buf(C::kWT ? 0 : ds), C::kWBytes, base, C::kSmem - 1024, 1024),
                              31)) {
                    if (rank == 0)
                        mbar_arrive_expect_tx(&bar_ready[ds], 2 * (bytes + (main_step ? 0 : C::kWBytes)));
                    const uint32_t bar = lead(&bar_ready[ds]);
                    if (main_step) {
                        const int kb = (tt.kb0 + it - main0(tt)) * C::kKS;
#pragma unroll
                        for (int h = 0; h < C::kKS; ++h)
#pragma unroll
                            for (int ms = 0; ms < C::kSubs; ++ms)
                                if (ms < tt.nsub)
                                    tma_load_2d_pair(t_buf(ds) + h * C::kTok + ms * C::kSub, &map_t.m[box[ms]], bar,
                                                     (kb + h) * 64, sub_row(tt, ms));
                    } else {
                        // [hi | lo] against the factor twice
                        const int half = tt.n_ext * C::kKS / 2;
                        if (!waited) {
                            grid_dependency_wait();
                            asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
                        }
                        waited = true;
#pragma unroll
                        for (int h = 0; h < C::kKS; ++h) {
                            const int j = j0 + h, jb = j % half;
#pragma unroll
                            for (int ms = 0; ms < C::kSubs; ++ms)
                                if (ms < tt.nsub)
                                    tma_load_2d_pair(t_buf(ds) + h * C::kTok + ms * C::kSub, &map_te.m[box[ms]], bar,
                                                     j * 64, sub_row(tt, ms));
                            uint8_t* dst = w_buf(C::kWT ? 0 : ds) + h * C::kW;
                            if constexpr (DX) {
#pragma unroll
                                for (int c = 0; c < C::kBM / 64; ++c)
                                    tma_load_3d_pair(dst + c * 8192, &map_we, bar, tt.h0 + c * 64, jb * 64, tt.g.e);
                            } else {
                                tma_load_3d_pair(dst, &map_we, bar, jb * 64, tt.h0, tt.g.e);
                            }
                        }
                    }
                }
                __syncwarp();
                if (++ds == DS) {
                    ds = 0;
                    done ^= 1u;
                }
                codes_step();
            }
        }
        // a pair without extension steps waits too, so that this grid's
        // completion implies that of the kernels before it
        if (!waited) grid_dependency_wait();
        if (stop) {
            // let the copies already issued land before the CTA exits (those
            // that complete in the other CTA: by time)
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < 1000000) {}
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ tensor memory, MMAs
        __syncwarp();  // the cluster barrier does not bring a warp's threads together
        tmem2_alloc(&s_tmem, C::kTmemCols);
        tc_fence_before();
        asm volatile("bar.arrive 2, %0;" ::"r"(32 + kWork) : "memory");
        __syncwarp();
        tc_fence_after();
        if (rank == 0) {
            // Everything here is uniform over the warp, and said to be (values that
            // went through a shuffle from lane 0), so that descriptors stay in
            // uniform registers and an MMA costs a few clocks to issue.
            const uint32_t tmem_d = __shfl_sync(0xFFFFFFFFu, s_tmem, 0);
            bool stop = false;
            int n_masked = 0, ds = 0;
            bool early = false;
            uint32_t ready = 0;
            Walk walk;
            first_tile(walk);
            const uint64_t w_desc0 = tile_desc(smem_u32(w_buf(0)), DX, 0);
            const uint64_t t_desc0 = tile_desc(smem_u32(t_buf(0)), false, 0);
            constexpr uint32_t kWk = DX ? 2048 / 16 : 32 / 16, kTk = 32 / 16;  // next 16 of the contraction
            for (int tl = 0; !stop; ++tl) {
                Tile t;
                if (!next_tile(walk, t)) break;
                const int nsub = __shfl_sync(0xFFFFFFFFu, t.nsub, 0);
                const int n_main = __shfl_sync(0xFFFFFFFFu, t.n_main, 0);
                const int n_iter = __shfl_sync(0xFFFFFFFFu, t.n_main + t.n_ext, 0);
                const int ext_last = DROP ? __shfl_sync(0xFFFFFFFFu, t.n_ext, 0) - 1 : -1;
                const uint32_t idesc0 = __shfl_sync(
                    0xFFFFFFFFu, C::kIdesc | (static_cast<uint32_t>(max(32, sub_n(t, 0)) >> 3) << 17), 0);
                const uint32_t idesc1 = __shfl_sync(
                    0xFFFFFFFFu, C::kIdesc | (static_cast<uint32_t>(max(32, sub_n(t, 1)) >> 3) << 17), 0);
                // the accumulators of the last tile that had them have been read
                const uint32_t acc_d = tmem_d + (C::kAccs == 2 ? (tl & 1) * C::kAccCols : 0);
                if (tl >= C::kAccs)
                    stop = !__all_sync(0xFFFFFFFFu, mbar_wait(&bar_free[tl % C::kAccs], (tl / C::kAccs + 1) & 1u,
                                                              abort_flag));
                for (int it = 0; it < n_iter && !stop; ++it) {
                    // the tokens and the weight tiles of both CTAs are in place; the
                    // next step's barrier is polled beside the MMAs' issue
                    if (!early) stop = !__all_sync(0xFFFFFFFFu, mbar_wait(&bar_ready[ds], ready, abort_flag));
                    if (stop) break;
                    tc_fence_after();
                    const bool wrap = ds + 1 == DS;
                    const bool next = mbar_test(&bar_ready[wrap ? 0 : ds + 1], wrap ? ready ^ 1u : ready);
                    const uint64_t td = t_desc0 + static_cast<uint32_t>(ds) * (C::kTokBytes / 16);
                    const uint32_t acc = it > 0 ? 1u : 0u;
                    if (C::kWT && it < n_main) {
                        const uint32_t wt = tmem_d + C::kAccs * C::kAccCols + ds * (32 * C::kKS);
#pragma unroll
                        for (int k = 0; k < 4 * C::kKS; ++k)
                            mma2_elect_ts(acc_d, wt + 8 * k, td + (k / 4) * (C::kTok / 16) + (k % 4) * kTk, idesc0,
                                          k > 0 ? 1u : acc);
                    } else {
                        const int ws = C::kWT ? 0 : ds;
                        const uint64_t wd = w_desc0 + static_cast<uint32_t>(ws) * (C::kWBytes / 16);
#pragma unroll
                        for (int h = 0; h < C::kKS; ++h) {
                            const uint64_t w64 = wd + h * (C::kW / 16), t64 = td + h * (C::kTok / 16);
                            mma2_elect4<kWk, kTk>(acc_d, w64, t64, idesc0, h > 0 ? 1u : acc);
                            if (C::kSubs == 2 && nsub == 2)
                                mma2_elect4<kWk, kTk>(acc_d + C::kSubT, w64, t64 + C::kSub / 16, idesc1,
                                                      h > 0 ? 1u : acc);
                        }
                    }
                    mma2_commit_elect(&bar_done[ds]);
                    early = __all_sync(0xFFFFFFFFu, next);
                    if (DROP && it == ext_last) {
                        mma2_commit_elect(&bar_ext);
                        stop = !__all_sync(0xFFFFFFFFu, mbar_wait(&bar_masked, n_masked++ & 1u, abort_flag));
                    }
                    if (++ds == DS) {
                        ds = 0;
                        ready ^= 1u;
                    }
                }
                mma2_commit_elect(&bar_accum[tl % C::kAccs]);
            }
        }
    } else if (C::kCodeWarp && warp == 2 + C::kWorkWarps) {
        // ------------------------------------------------------------ codes
        Tile t;
        Walk walk;
        first_tile(walk);
        int cs = 0;
        uint32_t freed = 0;
        bool stop = false;
        while (!stop && next_tile(walk, t)) {
            const int n_iter = t.n_main + t.n_ext;
            for (int it = 0; it < n_iter; ++it) {
                stop = __any_sync(0xFFFFFFFFu, !mbar_wait(&bar_cfree[cs], freed ^ 1u, abort_flag) || *abort_flag);
                if (stop) break;
                load_codes(t, it, cs);
                if (++cs == LC) {
                    cs = 0;
                    freed ^= 1u;
                }
            }
        }
        if (stop) {  // as above
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < 1000000) {}
        }
    } else {
        const int ew = warp - 2;
        const int q = warp & 3;  // tensor memory lane quadrant of this warp
        const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
        // tokens of an accumulator per warp, whole loads of 32 (so that some warps
        // have none where the tile is small)
        constexpr int kParts = C::kWorkWarps / 4;
        constexpr int kShare = C::kSubT / kParts < 32 ? 32 : C::kSubT / kParts;
        static_assert(kShare % 32 == 0 && (kShare * kParts == C::kSubT || C::kSubT == 32), "shares");
        const int tbeg = (ew / 4) * kShare;
        asm volatile("bar.sync 2, %0;" ::"r"(32 + kWork) : "memory");
        tc_fence_after();
        const uint32_t tmem_d = s_tmem;
        // ------------------------------------------------------------ keep and scale V A
        // this warp's part of the accumulators; n counts these calls
        auto mask_accumulators = [&](const Tile& t, int tl, int n) {
            grid_dependency_wait();  // the generator's state may be as young as V
            KeepGen gen;
            gen.init(args.drop);
            if (__all_sync(0xFFFFFFFFu, mbar_wait(&bar_ext, n & 1u, abort_flag))) {
                tc_fence_after();
                const int col = t.h0 + q * 32 + lane;
                for (int ms = 0; ms < t.nsub; ++ms) {
#pragma unroll 1
                    for (int tt = tbeg; tt < tbeg + kShare && ms * C::kSubT + tt < t.tokens; tt += 32) {
                        const uint32_t at = tmem_d + lane_base + tl % C::kAccs * C::kAccCols + ms * C::kSubT + tt;
                        uint32_t v[32];
                        tmem_ld_32x32b_x32(at, v);
                        tmem_ld_wait();
                        const int64_t row0 = t.g.row0 + ms * C::kSubT + tt;
#pragma unroll
                        for (int o = 0; o < 4; ++o) {
                            // the eight lanes of a generator group draw it for eight
                            // tokens, one each, and exchange the decisions
                            uint32_t f[4];
                            gen.flags(static_cast<uint64_t>((row0 + 8 * o + (lane & 7)) * args.cols + (col & ~7)) >> 3,
                                      f);
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
        const int team = ew / C::kTeamWarps;
        // a thread of kBM; with as many threads as a step has units, which 64 of it
        // (into tensor memory a warp writes the lanes of its own quadrant)
        const int dt = C::kWT ? q * 32 + lane : (threadIdx.x - 64) % C::kBM;
        const int half = C::kKS > C::kUnits ? (threadIdx.x - 64) / C::kBM % (C::kKS / C::kUnits) : 0;
        float level = 0.0f;  // of shuffle_word
#pragma unroll
        for (int i = 0; i < 16; ++i) level = (lane & 15) == i ? nf4_level(i) : level;
        const bool fp32_scales = args.absmax != nullptr;  // no double quantisation
        const float mu = fp32_scales ? 0.0f : __ldg(args.scale_mean);
        // This thread's unit of a step.  Forward: weight row h0 + dt, block kb.
        // Input gradient: weight row 64 kb + n_local, block cblk of this CTA's
        // columns, dealt so that the eight threads of a quarter warp store to
        // distinct bank groups and read codes at most two to one.
        constexpr int kCB = C::kBM / 64;
        static_assert(kCB == 2, "unit mapping");
        int n_local = dt, cblk = 0;
        if constexpr (DX) {
            const int qw = dt >> 3, i = dt & 7;
            n_local = 8 * (qw >> 1) + i;
            cblk = ((i >> 1) + qw) & 1;
        }
        int dst_off = half * C::kW + (DX ? cblk * 8192 + n_local * 128 + ((n_local & 7) << 4)
                                               : dt * 128 + ((dt & 7) << 4));
        int code_off = half * C::kCodes + (DX ? n_local * kCB + cblk : dt) * 32;
        if (!NF4_CHECK(code_off + (C::kUnits - 1) * C::kCodes + 32 <= C::kCBytes &&
                           (C::kWT || (dst_off | 0x70) + 16 + (C::kUnits - 1) * C::kW <= C::kWBytes),
                       38))
            code_off = dst_off = 0;
        // The units' block scales are fetched one own step (several steps of the
        // pair) ahead: an 8-bit code and the second-level scale, or the fp32 scale.
        // With few tokens and an even number of blocks per row a step's two scales
        // are one load, and share their second-level scale.  Every instruction here
        // is one that the decode's pipe has no time for, so that what depends on the
        // tile alone is worked out once for it (indices of blocks fit 32 bits).
        struct Scale {
            uint32_t ok;  // bit h: the unit lies inside the expert's weight
            int q[C::kUnits];
            float a2[C::kUnits];
        };
        constexpr bool kPairs = !DX && C::kUnits == 2;
        const bool pairs = kPairs && args.w_blocks_per_row % 2 == 0 &&
                           (fp32_scales ? (reinterpret_cast<uintptr_t>(args.absmax) & 7) == 0
                                        : (reinterpret_cast<uintptr_t>(args.qscale) & 1) == 0);
        const uint32_t k_blocks = DX ? C::kKS * 64 * static_cast<uint32_t>(args.w_blocks_per_row) : C::kKS;
        uint32_t block0 = 0;       // of the first unit in step 0 of tile t's contraction
        int k_end[C::kUnits] = {}; // unit h exists in the steps before this one
        auto enter = [&](const Tile& t) {
            const int kb = t.kb0 * C::kKS + half;
            const int row = DX ? kb * 64 + n_local : t.h0 + dt, blk = DX ? t.h0 / 64 + cblk : kb;
            block0 = (static_cast<uint32_t>(t.g.e) * args.w_rows + row) * args.w_blocks_per_row + blk;
            const bool inside = DX ? blk < args.w_blocks_per_row : row < args.w_rows;
            // 64s of the contraction that this thread's units have
            const int kbs = DX ? (args.w_rows - n_local + 63) >> 6 : args.w_blocks_per_row;
#pragma unroll
            for (int h = 0; h < C::kUnits; ++h)
                k_end[h] = inside ? min(t.n_main, (kbs - half - h + C::kKS - 1) / C::kKS - t.kb0) : 0;
        };
        // the encoded weight has this block's scales
        auto have_block = [&](uint32_t b) {
            return NF4_CHECK(b < static_cast<uint64_t>(args.E) * args.w_rows * args.w_blocks_per_row, 33);
        };
        auto fetch = [&](int k) {
            Scale s;
            s.ok = 0;
            const uint32_t b0 = block0 + static_cast<uint32_t>(k) * k_blocks;
            if (kPairs && pairs) {
                s.q[0] = 0;
                s.a2[0] = 0.0f;
                if (k < k_end[0] && have_block(b0) && have_block(b0 + 1)) {
                    s.ok = 1;
                    if (fp32_scales) {
                        const float2 two = __ldg(reinterpret_cast<const float2*>(args.absmax + b0));
                        s.a2[0] = two.x;
                        s.q[0] = __float_as_int(two.y);
                    } else {
                        s.q[0] = __ldg(reinterpret_cast<const short*>(args.qscale + b0));
                        s.a2[0] = __ldg(args.scale2 + (b0 >> 8));
                    }
                }
                return s;
            }
#pragma unroll
            for (int h = 0; h < C::kUnits; ++h) {
                s.q[h] = 0;
                s.a2[h] = 0.0f;
                const uint32_t b = b0 + (DX ? h * 64 * static_cast<uint32_t>(args.w_blocks_per_row) : h);
                if ((!DROP || k >= 0) && k < k_end[h] && have_block(b)) {
                    s.ok |= 1u << h;
                    if (fp32_scales) {
                        s.a2[h] = __ldg(args.absmax + b);
                    } else {
                        s.q[h] = __ldg(args.qscale + b);
                        s.a2[h] = __ldg(args.scale2 + (b >> 8));
                    }
                }
            }
            return s;
        };
        // ------------------------------------------------------------ epilogue of tile tl
        // Lane: weight column.  A pair of lanes swaps halves of two tokens' values,
        // so that a store writes two tokens' 64-byte runs (fp32 partials: 128 bytes
        // of one token).
        auto epilogue = [&](const Tile& t, int tl) {
            const bool done = mbar_wait(&bar_accum[tl % C::kAccs], tl / C::kAccs & 1u, abort_flag);
            const bool ok = __all_sync(0xFFFFFFFFu, done && !*abort_flag);
            tc_fence_after();
            const uint32_t odd = lane & 1, sel = odd ? 0x3276u : 0x5410u;
            const int col = t.h0 + q * 32 + lane, col2 = col & ~1;
            for (int ms = 0; ok && ms < t.nsub; ++ms) {
#pragma unroll 1
                for (int tt = tbeg; tt < tbeg + kShare && ms * C::kSubT + tt < t.tokens; tt += 32) {
                    __syncwarp();  // the lanes' stores differ; tensor memory is read by the whole warp
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(tmem_d + lane_base + tl % C::kAccs * C::kAccCols + ms * C::kSubT + tt, v);
                    tmem_ld_wait();
                    const int at = ms * C::kSubT + tt, left = t.tokens - at;
                    if (args.splits > 1) {
                        float* dst = args.part + (static_cast<int64_t>(t.z) * args.M + t.g.row0 + at) * args.cols + col;
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            if (T <= 64 && j % 8 == 0 && j >= left) break;
                            if (j < left && col < args.cols &&
                                NF4_CHECK(in_span(dst + static_cast<int64_t>(j) * args.cols, 4, args.part,
                                                  static_cast<int64_t>(args.splits) * args.M * args.cols * 4, 4),
                                          34))
                                dst[static_cast<int64_t>(j) * args.cols] = __uint_as_float(v[j]);
                        }
                    } else {
                        uint16_t* dst = args.out + static_cast<int64_t>(t.g.row0 + at + odd) * args.cols + col2;
                        // cols is a multiple of 8
                        const int rows = col2 < args.cols ? left - static_cast<int>(odd) : 0;
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            if (T <= 64 && j % 8 == 0 && j >= left) break;
                            const uint32_t own = pack_bf16x2(__uint_as_float(v[j]), __uint_as_float(v[j + 1]));
                            const uint32_t two = __byte_perm(own, __shfl_xor_sync(0xFFFFFFFFu, own, 1), sel);
                            if (j < rows && NF4_CHECK(in_span(dst + static_cast<int64_t>(j) * args.cols, 4, args.out,
                                                              static_cast<int64_t>(args.M) * args.cols * 2, 4),
                                                      35))
                                *reinterpret_cast<uint32_t*>(dst + static_cast<int64_t>(j) * args.cols) = two;
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_pair(lead(&bar_free[tl % C::kAccs]));
            return ok;
        };

        Tile t;
        Walk walk;
        first_tile(walk);
        bool have = next_tile(walk, t);
        // this team's next step: its place in tile t, its slots and the parities of
        // the rounds over them
        int it = team, ds = team, cs = team, n_masked = 0;
        uint32_t cp = 0, dp = 1;
        const uint32_t ready0 = lead(&bar_ready[0]);
        Scale ahead{};
        if (have) {
            enter(t);
            ahead = fetch(it - main0(t));
        }
        // A tile's results go out once this team has its first steps of the next
        // tile in place, so that the MMAs never wait for a decode there.
        constexpr int kDefer = DS / C::kTeams;
        Tile last;             // the tile whose results are still to go out, if any
        bool pending = false, masked = !DROP || t.n_ext == 0;
        int tl = 0, own = -1;  // own: with a tile pending, this team's steps of tile t so far
        int n_iter = t.n_main + t.n_ext;
#pragma unroll 1
        while (true) {
            const bool ended = !have || it >= n_iter;
            if (ended || own == kDefer || (DROP && !masked)) {
                const bool mask_now = DROP && !masked && (ended || is_main(t, it)) && have;
                if (pending && (ended || own == kDefer || mask_now)) {
                    if (!epilogue(last, tl - 1)) break;
                    pending = false;
                    own = -1;
                }
                if (!have) break;
                if (mask_now) {
                    masked = true;
                    mask_accumulators(t, tl, n_masked++);
                }
                if (ended) {
                    last = t;
                    pending = true;
                    own = 0;
                    it -= n_iter;
                    have = next_tile(walk, t);
                    ++tl;
                    if (have) {
                        enter(t);
                        ahead = fetch(it - main0(t));
                        masked = !DROP || t.n_ext == 0;
                        n_iter = t.n_main + t.n_ext;
                    }
                    continue;
                }
            }
            const bool main_step = is_main(t, it);
            float sc[C::kUnits];
            if (kPairs && pairs) {
                if (fp32_scales) {
                    sc[0] = ahead.a2[0];
                    sc[C::kUnits - 1] = __int_as_float(ahead.q[0]);
                } else {
#pragma unroll
                    for (int h = 0; h < C::kUnits; ++h)
                        sc[h] = ahead.ok ? nf4_block_scale(static_cast<int8_t>(ahead.q[0] >> 8 * h), ahead.a2[0], mu)
                                         : 0.0f;
                }
            } else {
#pragma unroll
                for (int h = 0; h < C::kUnits; ++h)
                    sc[h] = !(ahead.ok >> h & 1u) ? 0.0f
                            : fp32_scales         ? ahead.a2[h]
                                                  : nf4_block_scale(static_cast<int8_t>(ahead.q[h]), ahead.a2[h], mu);
            }
            // two polls whose latencies overlap; bounded waits where one is early
            const bool both = mbar_try_wait(&bar_codes[cs], cp) & mbar_try_wait(&bar_done[ds], dp);
            const bool ok =
                both || (mbar_wait(&bar_codes[cs], cp, abort_flag) && mbar_wait(&bar_done[ds], dp, abort_flag));
            if (__any_sync(0xFFFFFFFFu, !ok)) break;  // the warp stays together
            it += C::kTeams;
            ahead = fetch(it - main0(t));
            if (!NF4_CHECK(cs < LC && ds < DS, 36)) break;  // of the whole warp
            // a unit outside the weight has a zero scale and decodes to zeros
            if (C::kWT && main_step) {
                tc_fence_after();
#pragma unroll 1  // less code to fetch for short calls: 500 tokens over 64 experts 78.5 to 76.7 us
                for (int h = 0; h < C::kUnits; ++h)
                    decode_lane(codes_buf(cs) + h * C::kCodes + code_off, h ? sc[C::kUnits - 1] : sc[0], level,
                                tmem_d + lane_base + C::kAccs * C::kAccCols + (ds * C::kKS + h + half) * 32);
                tmem_st_wait();
                tc_fence_before();
            } else if (main_step) {
#pragma unroll 1
                for (int h = 0; h < C::kUnits; ++h)
                    decode_row<(T <= 256)>(codes_buf(cs) + h * C::kCodes + code_off, h ? sc[C::kUnits - 1] : sc[0],
                                           level, w_buf(ds) + h * C::kW + dst_off);
            }
            if (!C::kWT) fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (C::kCodeWarp) mbar_arrive(&bar_cfree[cs]);
                mbar_arrive_pair(ready0 + 8 * ds);
            }
            if (own >= 0) ++own;
            cs += C::kTeams;
            if (cs >= LC) {
                cs -= LC;
                cp ^= 1u;
            }
            ds += C::kTeams;
            if (ds >= DS) {
                ds -= DS;
                dp ^= 1u;
            }
        }
    }
    // neither CTA frees its tensor memory or leaves while the other may still
    // use it, read its operands or arrive on its barriers
    __syncwarp();
    tc_fence_before();
    cluster_arrive_release();
    cluster_wait_acquire();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem2_dealloc(s_tmem, C::kTmemCols);
    }
}

// out [M, cols] = the splits' partials added in order; rows outside the groups
// are left as they are.  cols is a multiple of 8.
__global__ void k_group_sum(const int32_t* offsets, int E, int M, int cols, int splits, const float* __restrict__ part,
                            uint16_t* __restrict__ out) {
    grid_dependency_wait();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int lo = 0, hi = M;
    if (offsets != nullptr) {
        lo = min(max(__ldcg(offsets), 0), M);
        hi = min(max(__ldcg(offsets + E), lo), M);
    }
    const int quads = cols / 4;
    const int64_t total = static_cast<int64_t>(hi - lo) * quads, slice = static_cast<int64_t>(M) * quads;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const float4* p = reinterpret_cast<const float4*>(part) + static_cast<int64_t>(lo) * quads + i;
        if (!NF4_CHECK(in_span(p + (splits - 1) * slice, 16, part, splits * slice * 16, 16) &&
                           in_span(out + 4 * (static_cast<int64_t>(lo) * quads + i), 8, out, slice * 8, 8),
                       37))
            continue;
        float4 v = __ldcg(p);
        for (int z = 1; z < splits; ++z) {
            const float4 x = __ldcg(p + z * slice);
            v.x += x.x;
            v.y += x.y;
            v.z += x.z;
            v.w += x.w;
        }
        reinterpret_cast<uint2*>(out)[static_cast<int64_t>(lo) * quads + i] =
            make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    }
}

}  // namespace nf4lora
