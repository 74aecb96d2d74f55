// Host orchestration of the NF4-LoRA layer with adapter dropout and of the
// layer of a mixture of experts (kernels: grouped.cuh, rank.cuh; formulas
// there).  Both are the same chain; the dense layer is one group of all rows.
//
//   forward   rank T -> sum (pair of T) -> fused product
//   backward  rank V -> sum (pair of V) -> fused input gradient
//             -> pair of the saved T -> dB -> dA
//
// Every kernel is a programmatic dependent of the one before it and waits for
// it first, except the fused products, which wait only before they read the
// pair: what else they read was complete before the sum started.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "adapter.h"
#include "group_plan.h"
#include "grouped.cuh"
#include "kernels.h"
#include "rank.cuh"
#include "trace.h"

namespace nf4lora {

namespace {

thread_local cudaError_t t_error = cudaSuccess;
cudaError_t keep(cudaError_t e) {
    if (e != cudaSuccess) t_error = e;
    return e;
}

int64_t up256(int64_t b) { return (b + 255) & ~int64_t(255); }

// ------------------------------------------------------------------ tensor maps
// [experts][rows][inner] with rows `ld` bytes apart and experts `rows` rows
// apart (experts 0: a plain matrix).  Reads outside give zeros.
bool make_map(CUtensorMap* m, CUtensorMapDataType type, int elem_bytes, const void* ptr, int64_t inner, int64_t rows,
              int64_t experts, uint32_t box_inner, uint32_t box_rows, CUtensorMapSwizzle swizzle) {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    if (!fn) return false;
    const int rank = experts > 0 ? 3 : 2;
    const cuuint64_t ld = static_cast<cuuint64_t>(inner) * elem_bytes;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows),
                          static_cast<cuuint64_t>(experts)};
    cuuint64_t strides[2] = {ld, ld * static_cast<cuuint64_t>(rows)};
    cuuint32_t box[3] = {box_inner, box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, type, rank, const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool map16(CUtensorMap* m, const void* ptr, int64_t inner, int64_t rows, int64_t experts, uint32_t box_rows) {
    return make_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, ptr, inner, rows, experts, 64, box_rows,
                    CU_TENSOR_MAP_SWIZZLE_128B);
}

bool map_packed(CUtensorMap* m, const uint8_t* codes, int64_t N, int64_t K, int64_t experts, uint32_t box_inner,
                uint32_t box_rows, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_NONE) {
    return make_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, codes, K / 2, N, experts, box_inner, box_rows, swizzle);
}

// ------------------------------------------------------------------ launches
// Opt-in to `smem` bytes of dynamic shared memory, once per kernel and device
// (kept out of stream captures after the first call).
cudaError_t opt_in(const void* kernel, int smem, bool (&done)[64]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                 cudaSharedmemCarveoutMaxShared);
    if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
    return e;
}

// A programmatic dependent of the kernel before it on the stream, in clusters
// of `cluster` CTAs along grid.x.
template <typename Kern, typename... Args>
cudaError_t launch_clustered(const char* name, Kern kern, dim3 grid, int cluster, int threads, int smem,
                             cudaStream_t st, const Args&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    TraceScope trace(name, st);
    return keep(cudaLaunchKernelEx(&cfg, kern, args...));
}

template <typename Kern, typename... Args>
cudaError_t launch_dependent(const char* name, Kern kern, dim3 grid, int threads, int smem, cudaStream_t st,
                             const Args&... args) {
    return launch_clustered(name, kern, grid, 1, threads, smem, st, args...);
}

dim3 flat_grid(int64_t items, int num_sms) {
    return dim3(static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(div_up(items, 256), num_sms * 8))));
}

// ------------------------------------------------------------------ workspaces
struct Workspace {
    uint16_t *T2, *V2, *B8;
    float *part, *fused_part;
    int64_t bytes;
};

Workspace layout(uint8_t* base, int64_t M, int E, int64_t N, int64_t K, int r, int num_sms, bool backward) {
    Workspace w{};
    int64_t off = 0;
    auto take = [&](int64_t bytes) {
        uint8_t* p = base ? base + off : nullptr;
        off += up256(bytes);
        return p;
    };
    const int64_t pair = M * 2 * rank64(r) * 2, rn = rank_width(r);
    w.T2 = reinterpret_cast<uint16_t*>(take(pair));
    if (backward) w.V2 = reinterpret_cast<uint16_t*>(take(pair));
    if (r % 8 != 0) w.B8 = reinterpret_cast<uint16_t*>(take(E * N * ceil_to(r, 8) * 2));
    int64_t part = rows_split(E, M, K, r, num_sms).splits * M * rn;
    if (backward) {
        part = std::max(part, rows_split(E, M, N, r, num_sms).splits * M * rn);
        part = std::max(part, most_partials(E, M, grad_part_steps(E, M, N, num_sms)) * N * rn);
        part = std::max(part, most_partials(E, M, grad_part_steps(E, M, K, num_sms)) * K * rn);
    }
    w.part = reinterpret_cast<float*>(take(part * 4));
    // apart from the rank-r partials, whose sum may still run when the fused
    // product's first tiles end
    const int64_t cols = backward ? K : N;
    const FusedPlan f = plan_fused(backward, E, M, cols, backward ? N : K, r, num_sms);
    if (f.splits > 1) w.fused_part = reinterpret_cast<float*>(take(f.splits * M * cols * 4));
    w.bytes = off;
    return w;
}

// ------------------------------------------------------------------ rank-r products
// B with its rows padded to a multiple of eight elements (16 bytes, as tensor
// maps need).
__global__ void k_pad_columns(const uint16_t* __restrict__ src, int64_t rows, int cols, int padded,
                              uint16_t* __restrict__ dst) {
    grid_dependency_wait();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t total = rows * padded;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t row = i / padded;
        const int c = static_cast<int>(i - row * padded);
        dst[i] = c < cols ? src[row * cols + c] : uint16_t(0);
    }
}

template <int MODE, bool DROP>
cudaError_t launch_rank(const char* name, const CUtensorMap& a, const CUtensorMap& b, RankArgs g, dim3 grid,
                        cudaStream_t st) {
    using C = RankConfig<MODE, DROP>;
    constexpr bool tok = C::kTok;
    const int rchunks = (g.rn + 63) / 64;
    g.a_bytes = tok ? 4 * 8192 : 16384;
    g.b_bytes = tok ? 2 * rchunks * 8192 : MODE == RANK_V ? rchunks * 8192 : g.rn * 128;
    const int slot = g.a_bytes + g.b_bytes;
    // half an SM's shared memory where that holds two stages, else what one CTA
    // can have
    int stages = std::min(kRankStages, 111 * 1024 / slot);
    if (stages < 2) stages = std::min(kRankStages, 224 * 1024 / slot);
    g.stages = stages;
    const int sets = tok ? 2 : static_cast<int>(div_up(g.k_per_split, g.run_steps)), cols = sets * g.rn;
    g.tmem_cols = 32;
    while (g.tmem_cols < cols) g.tmem_cols *= 2;
    // CTAs that share an SM must not wait for each other's tensor memory
    if (g.tmem_cols > 256 && 2 * (stages * slot + 1024) <= 226 * 1024) return keep(cudaErrorInvalidConfiguration);
    static bool done[64] = {};
    const cudaError_t e = opt_in(reinterpret_cast<const void*>(&k_rank<MODE, DROP>), 226 * 1024, done);
    if (e != cudaSuccess) return keep(e);
    return launch_dependent(name, k_rank<MODE, DROP>, grid, C::kThreads, stages * slot + 1024, st, a, b, g);
}

RankArgs rank_args(const GroupCtx& c) {
    RankArgs g{};
    g.offsets = c.offsets;
    g.E = c.E;
    g.M = static_cast<int>(c.M);
    g.r = c.r;
    g.rn = rank_width(c.r);
    g.r64 = rank64(c.r);
    g.drop = c.drop;
    g.drop_cols = static_cast<int>(c.K);
    return g;
}

// The pair of T (act X, factor A) or V (act dY, factor B): the product in
// splits, then their sum.
int rank_rows(const GroupCtx& c, bool is_t, const uint16_t* act, const uint16_t* factor, uint16_t* pair, float* out32,
              float* part) {
    const int64_t contraction = is_t ? c.K : c.N;
    const GroupSplit sp = rows_split(c.E, c.M, contraction, c.r, c.num_sms);
    RankArgs g = rank_args(c);
    g.check = c.offsets != nullptr ? 1 : 0;
    g.k_steps = static_cast<int>(div_up(contraction, 64));
    g.k_per_split = sp.per;
    g.run_steps = static_cast<int>(std::min<int64_t>(kRunSteps, std::max<int64_t>(4, div_up(sp.per, rank_sets(c.r)))));
    g.part = part;
    g.part_slice = c.M * g.rn;
    CUtensorMap ma, mb;
    std::memset(&ma, 0, sizeof(ma));
    std::memset(&mb, 0, sizeof(mb));
    if (!map16(&ma, act, contraction, c.M, 0, 128)) return -1;
    if (is_t ? !map16(&mb, factor, c.K, c.r, c.E, g.rn) : !map16(&mb, factor, ceil_to(c.r, 8), c.N, c.E, 64)) return -1;
    const dim3 grid(static_cast<unsigned>(most_tiles(c.offsets != nullptr, c.E, c.M, 128)), 1, sp.splits);
    const bool drop = is_t && c.drop.threshold != 0;
    g.alpha = drop ? c.s * c.drop.gain : c.s;
    if (sp.splits == 1) {
        g.pair = pair;
        g.out32 = out32;
    }
    const cudaError_t e = drop   ? launch_rank<RANK_T, true>("rank_t_drop", ma, mb, g, grid, c.stream)
                          : is_t ? launch_rank<RANK_T, false>("rank_t", ma, mb, g, grid, c.stream)
                                 : launch_rank<RANK_V, false>("rank_v", ma, mb, g, grid, c.stream);
    if (e != cudaSuccess) return -2;
    if (sp.splits == 1) return 0;
    RankRowsSumArgs s{};
    s.offsets = c.offsets;
    s.E = c.E;
    s.M = g.M;
    s.part = part;
    s.splits = sp.splits;
    s.slice = g.part_slice;
    s.r = c.r;
    s.rn = g.rn;
    s.r64 = g.r64;
    s.alpha = g.alpha;
    s.pair = pair;
    s.out32 = out32;
    return launch_dependent("rank_sum", k_rank_rows_sum, flat_grid(c.M * (g.r64 / 8), c.num_sms), 256, 0, c.stream,
                            s) == cudaSuccess ? 0 : -2;
}

// dB (act dY, pair T2) or dA (act X, pair V2).  late_wait: the pair was complete
// before the kernel launched last released its dependents.  check: no T or V kernel
// of this call has looked at the offsets.
int rank_grad(const GroupCtx& c, bool is_b, const uint16_t* act, const uint16_t* pair, uint16_t* out, int accumulate,
              bool late_wait, bool check, float* part) {
    const int64_t rows = is_b ? c.N : c.K;
    const int part_steps = grad_part_steps(c.E, c.M, rows, c.num_sms);
    const int64_t parts = most_parts(c.M, part_steps);
    const bool drop = !is_b && c.drop.threshold != 0;
    RankArgs g = rank_args(c);
    g.check = check && c.offsets != nullptr ? 1 : 0;
    g.rows = static_cast<int>(rows);
    g.part_steps = part_steps;
    g.slots = static_cast<int>(most_partials(c.E, c.M, part_steps));
    g.alpha = drop ? c.drop.gain : 1.0f;
    g.part = part;
    g.part_slice = rows * g.rn;
    g.out = out;
    g.accumulate = accumulate;
    g.late_wait = late_wait ? 1 : 0;
    CUtensorMap ma, mb;
    std::memset(&ma, 0, sizeof(ma));
    std::memset(&mb, 0, sizeof(mb));
    if (!map16(&ma, act, rows, c.M, 0, 64) || !map16(&mb, pair, 2 * g.r64, c.M, 0, 64)) return -1;
    const dim3 grid(static_cast<unsigned>(div_up(rows, 256)),
                    static_cast<unsigned>(c.E == 1 ? parts : c.E + most_partials(c.E, c.M, part_steps)));
    const cudaError_t e = is_b   ? launch_rank<RANK_DB, false>("rank_db", ma, mb, g, grid, c.stream)
                          : drop ? launch_rank<RANK_DA, true>("rank_da_drop", ma, mb, g, grid, c.stream)
                                 : launch_rank<RANK_DA, false>("rank_da", ma, mb, g, grid, c.stream);
    if (e != cudaSuccess) return -2;
    if (parts == 1) return 0;
    const bool vec = !is_b || c.r % 4 == 0;
    const int64_t sum_blocks = c.E * div_up(rows * c.r / (vec ? 4 : 1), 256);
    const dim3 sum_grid(static_cast<unsigned>(std::min<int64_t>(sum_blocks, 4 * c.num_sms)));
    const int cap = std::max(1, std::min(c.E, g.slots / 2));
    auto sum = [&](auto kern) {
        return launch_dependent("rank_grad_sum", kern, sum_grid, 256, cap * kSumGroupBytes, c.stream, c.offsets, c.E,
                                g.M, part_steps, g.slots, static_cast<const float*>(part), static_cast<int>(rows), c.r,
                                g.rn, g.alpha, out, accumulate, cap);
    };
    return (!is_b ? sum(k_rank_grad_sum<true, 4>)
            : vec ? sum(k_rank_grad_sum<false, 4>)
                  : sum(k_rank_grad_sum<false, 1>)) == cudaSuccess ? 0 : -2;
}

// ------------------------------------------------------------------ fused products
// m: the maps of k_group_gemm, those of the tokens (0 and 2) still to be made.
struct FusedMaps {
    RowMaps act_rows, pair_rows;
    CUtensorMap codes, factor;
    const uint16_t *act, *pair;
    int64_t contraction, pair_cols, M;
};

template <bool DX, int T, bool DROP>
cudaError_t launch_group_gemm(const char* name, FusedMaps& f, GroupGemmArgs g, bool cols_fastest, int num_sms,
                              bool* mapped, cudaStream_t st) {
    using C = GroupGemmConfig<DX, T>;
    static bool done[64] = {};
    const cudaError_t e = opt_in(reinterpret_cast<const void*>(&k_group_gemm<DX, T, DROP>), C::kSmem, done);
    if (e != cudaSuccess) return keep(e);
    *mapped = true;
    for (int i = 0; i < C::kBoxes; ++i)
        *mapped = *mapped && map16(&f.act_rows.m[i], f.act, f.contraction, f.M, 0, C::kBoxRows * (i + 1)) &&
                  map16(&f.pair_rows.m[i], f.pair, f.pair_cols, f.M, 0, C::kBoxRows * (i + 1));
    if (!*mapped) return cudaSuccess;
    const int64_t row_tiles = most_tiles(g.offsets != nullptr, g.E, g.M, g.tile_rows);
    g.row_tiles = cols_fastest ? -1 : static_cast<int>(row_tiles);
    g.most_row_tiles = static_cast<int>(row_tiles);
    // one CTA (or two) on every SM, each pair walking its share of the tiles
    const int64_t pairs =
        std::min<int64_t>(num_sms / 2 * C::kMinBlocks, row_tiles * g.col_tiles * g.splits);
    const int fast = g.row_tiles >= 0 ? g.row_tiles : g.col_tiles;
    g.walk_z = static_cast<int>(pairs % g.splits);
    g.walk_fast = static_cast<int>(pairs / g.splits % fast);
    g.walk_slow = static_cast<int>(pairs / g.splits / fast);
    const dim3 grid(static_cast<unsigned>(2 * pairs));
    return launch_clustered(name, k_group_gemm<DX, T, DROP>, grid, 2, C::kThreads, C::kSmem, st, f.act_rows,
                            f.codes, f.pair_rows, f.factor, g);
}

// Y (act X, pair T2, factor B) or dX (act dY, pair V2, factor A).
int fused(const GroupCtx& c, bool dx, const uint16_t* act, const uint16_t* pair, const uint16_t* factor, float* part,
          uint16_t* out) {
    const int64_t contraction = dx ? c.N : c.K, cols = dx ? c.K : c.N;
    const int r64 = rank64(c.r);
    const FusedPlan plan = plan_fused(dx, c.E, c.M, cols, contraction, c.r, c.num_sms);
    GroupGemmArgs g{};
    g.offsets = c.offsets;
    g.E = c.E;
    g.M = static_cast<int>(c.M);
    g.cols = static_cast<int>(cols);
    g.k_main = plan.k_main;
    g.k_ext = plan.k_ext;
    g.splits = plan.splits;
    g.tile_rows = plan.tile_rows;
    g.col_tiles = static_cast<int>(div_up(cols, 256));
    g.qscale = c.qscale;
    g.scale2 = c.scale2;
    g.scale_mean = c.scale_mean;
    g.absmax = c.absmax;
    g.w_rows = static_cast<int>(c.N);
    g.w_blocks_per_row = static_cast<int>(c.K / 64);
    g.out = out;
    g.part = part;
    g.drop = c.drop;
    FusedMaps f;
    std::memset(&f, 0, sizeof(f));
    f.act = act;
    f.pair = pair;
    f.contraction = contraction;
    f.pair_cols = 2 * r64;
    f.M = c.M;
    if (dx ? !map_packed(&f.codes, c.codes, c.N, c.K, c.E, 64, 64) || !map16(&f.factor, factor, c.K, c.r, c.E, 64)
           : !map_packed(&f.codes, c.codes, c.N, c.K, c.E, 32, 128) ||
                 !map16(&f.factor, factor, ceil_to(c.r, 8), c.N, c.E, 128))
        return -1;
    // The tiles that run together share what they re-read.  Column tiles
    // fastest reads the activations once and a group's weight once per token
    // tile of that group, from L2 where the weight fits it; one dense weight
    // that does not goes token tiles fastest unless the activations are larger.
    const bool cols_fastest = c.offsets != nullptr || 2 * c.M * contraction > c.N * c.K * 33 / 64;
    const bool drop = dx && c.drop.threshold != 0;
    bool mapped = false;
    auto go = [&](auto dir, auto t) {
        constexpr bool DX = decltype(dir)::value;
        constexpr int T = decltype(t)::value;
        if constexpr (DX)
            if (drop)
                return launch_group_gemm<true, T, true>("group_gemm_dx_drop", f, g, cols_fastest, c.num_sms, &mapped,
                                                        c.stream);
        return launch_group_gemm<DX, T, false>(DX ? "group_gemm_dx" : "group_gemm_fwd", f, g, cols_fastest, c.num_sms,
                                               &mapped, c.stream);
    };
    auto pick = [&](auto dir) {
        constexpr int kFew = decltype(dir)::value ? 32 : 64;
        return plan.tile == kFew  ? go(dir, std::integral_constant<int, kFew>())
               : plan.tile == 256 ? go(dir, std::integral_constant<int, 256>())
                                  : go(dir, std::integral_constant<int, 512>());
    };
    cudaError_t e = dx ? pick(std::true_type()) : pick(std::false_type());
    if (e != cudaSuccess) return -2;
    if (!mapped) return -1;
    if (plan.splits > 1) {
        e = launch_dependent("group_sum", k_group_sum, flat_grid(c.M * cols / 4, c.num_sms), 256, 0, c.stream,
                             c.offsets, c.E, static_cast<int>(c.M), static_cast<int>(cols), plan.splits,
                             static_cast<const float*>(part), out);
        if (e != cudaSuccess) return -2;
    }
    return 0;
}

// B as the tensor maps can read it: itself, or its padded copy.
int padded_b(const GroupCtx& c, const uint16_t*& B, uint16_t* B8) {
    if (B8 == nullptr) return 0;
    const int r8 = static_cast<int>(ceil_to(c.r, 8));
    const int64_t rows = int64_t(c.E) * c.N;
    if (launch_dependent("pad_b", k_pad_columns, flat_grid(rows * r8, c.num_sms), 256, 0, c.stream, B, rows, c.r, r8,
                         B8) != cudaSuccess)
        return -2;
    B = B8;
    return 0;
}

}  // namespace

cudaError_t group_last_cuda_error() {
    const cudaError_t e = t_error;
    t_error = cudaSuccess;
    return e;
}

int64_t group_fwd_workspace_bytes(int64_t M, int E, int64_t N, int64_t K, int r, int num_sms) {
    return layout(nullptr, M, E, N, K, r, num_sms, false).bytes;
}
int64_t group_bwd_workspace_bytes(int64_t M, int E, int64_t N, int64_t K, int r, int num_sms) {
    return layout(nullptr, M, E, N, K, r, num_sms, true).bytes;
}

int group_fwd(const GroupCtx& c, const uint16_t* A, const uint16_t* B, const uint16_t* X, uint16_t* Y, float* T_saved,
              uint8_t* ws) {
    const Workspace w = layout(ws, c.M, c.E, c.N, c.K, c.r, c.num_sms, false);
    int rc = padded_b(c, B, w.B8);
    if (rc == 0) rc = rank_rows(c, true, X, A, w.T2, T_saved, w.part);
    if (rc == 0) rc = fused(c, false, X, w.T2, B, w.fused_part, Y);
    return rc;
}

int group_bwd(const GroupCtx& c, const uint16_t* A, const uint16_t* B, const uint16_t* X, const float* T_saved,
              const uint16_t* dY, uint16_t* dX, uint16_t* dA, uint16_t* dB, int accumulate, uint8_t* ws) {
    const Workspace w = layout(ws, c.M, c.E, c.N, c.K, c.r, c.num_sms, true);
    const bool need_v = dX != nullptr || dA != nullptr, have_t = T_saved != nullptr;
    int rc = 0;
    // The pair of T first: dB, which follows V or dX, then finds it complete and
    // starts beside their last CTAs; dA finds V complete behind dX.
    if (dB != nullptr && have_t) {
        const int r64 = rank64(c.r);
        if (launch_dependent("rank_pair", k_rank_pair, flat_grid(c.M * (r64 / 8), c.num_sms), 256, 0, c.stream, T_saved,
                             c.M, c.r, r64, w.T2) != cudaSuccess)
            rc = -2;
    }
    if (rc == 0 && need_v) {
        rc = padded_b(c, B, w.B8);
        if (rc == 0) rc = rank_rows(c, false, dY, B, w.V2, nullptr, w.part);
    }
    if (rc == 0 && dX != nullptr) rc = fused(c, true, dY, w.V2, A, w.fused_part, dX);
    if (rc == 0 && dB != nullptr) {
        if (!have_t) rc = rank_rows(c, true, X, A, w.T2, nullptr, w.part);
        if (rc == 0) rc = rank_grad(c, true, dY, w.T2, dB, accumulate, have_t && need_v, have_t && !need_v, w.part);
    }
    if (rc == 0 && dA != nullptr) rc = rank_grad(c, false, X, w.V2, dA, accumulate, dX != nullptr, false, w.part);
    return rc;
}

}  // namespace nf4lora
