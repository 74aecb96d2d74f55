// lora_dropout: out_i = keep_i x_i / (1 - p) over a flat array, the keep
// decisions from the counter-based generator of philox.cuh.  The gradient is
// the same call on the incoming gradient: no mask is written or read.
//
// Bound: HBM, an array in and an array out (8192 x 11008 bf16: 67 us, 5.4 TB/s,
// whatever the unrolling and the grid; one row of 4096: 2.9 us, the launch).  One
// thread takes whole groups of
// eight elements (16 bytes of bf16, 32 of fp32), kUnroll at a time with all
// their loads issued first, so that the generator's integer work (about 60
// instructions a group) runs while they are in flight.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "adapter.h"
#include "common.cuh"
#include "philox.cuh"
#include "trace.h"

namespace nf4lora {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

__device__ __forceinline__ uint32_t drop_pair(uint32_t x, uint32_t flags, float gain) {
    const float lo = __uint_as_float(x << 16), hi = __uint_as_float(x & 0xFFFF0000u);
    return pack_bf16x2((flags & 0x8000u) ? lo * gain : 0.0f, (flags >> 31) ? hi * gain : 0.0f);
}

__device__ __forceinline__ float4 drop_quad(float4 x, uint32_t f0, uint32_t f1, float gain) {
    return make_float4((f0 & 0x8000u) ? x.x * gain : 0.0f, (f0 >> 31) ? x.y * gain : 0.0f,
                       (f1 & 0x8000u) ? x.z * gain : 0.0f, (f1 >> 31) ? x.w * gain : 0.0f);
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) k_lora_dropout(const void* in, int64_t n, DropArgs drop, void* out) {
    constexpr int kVec = BF16 ? 1 : 2;  // 16-byte pieces of a group
    KeepGen gen;
    gen.init(drop);
    const int64_t groups = n / 8;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const uint4* src = static_cast<const uint4*>(in);
    uint4* dst = static_cast<uint4*>(out);
    for (int64_t g0 = first; g0 < groups; g0 += stride * kUnroll) {
        uint4 v[kUnroll][kVec];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (g0 + u * stride < groups)
#pragma unroll
                for (int h = 0; h < kVec; ++h) v[u][h] = __ldcs(src + (g0 + u * stride) * kVec + h);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t g = g0 + u * stride;
            if (g < groups && NF4_CHECK(in_span(src + g * kVec, 16 * kVec, in, n * (BF16 ? 2 : 4), 16) &&
                                            in_span(dst + g * kVec, 16 * kVec, out, n * (BF16 ? 2 : 4), 16),
                                        40)) {
                uint32_t f[4];
                gen.flags(static_cast<uint64_t>(g), f);
                if constexpr (BF16) {
                    const uint4 x = v[u][0];
                    __stcs(dst + g, make_uint4(drop_pair(x.x, f[0], drop.gain), drop_pair(x.y, f[1], drop.gain),
                                               drop_pair(x.z, f[2], drop.gain), drop_pair(x.w, f[3], drop.gain)));
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float4 x = *reinterpret_cast<const float4*>(&v[u][h]);
                        const float4 y = drop_quad(x, f[2 * h], f[2 * h + 1], drop.gain);
                        __stcs(reinterpret_cast<float4*>(dst) + 2 * g + h, y);
                    }
                }
            }
        }
    }
    // the last n % 8 elements, one thread each
    if (first < n % 8) {
        uint32_t f[4];
        gen.flags(static_cast<uint64_t>(groups), f);
        const int e = static_cast<int>(first);
        const int64_t i = 8 * groups + e;
        const uint32_t w = e < 4 ? (e < 2 ? f[0] : f[1]) : (e < 6 ? f[2] : f[3]);
        const bool keep = ((w >> ((e & 1) ? 31 : 15)) & 1u) != 0;
        if constexpr (BF16) {
            const float x = bf16_bits_to_float(static_cast<const uint16_t*>(in)[i]);
            const __nv_bfloat16 h = __float2bfloat16_rn(keep ? x * drop.gain : 0.0f);
            static_cast<uint16_t*>(out)[i] = *reinterpret_cast<const uint16_t*>(&h);
        } else {
            const float x = static_cast<const float*>(in)[i];
            static_cast<float*>(out)[i] = keep ? x * drop.gain : 0.0f;
        }
    }
}

}  // namespace

cudaError_t launch_lora_dropout(const void* in, int64_t n, bool bf16, const DropArgs& drop, void* out, int num_sms,
                                cudaStream_t stream) {
    const int64_t per_cta = int64_t(kThreads) * kUnroll;
    int64_t grid = (n / 8 + per_cta - 1) / per_cta;
    grid = std::max<int64_t>(1, std::min<int64_t>(grid, int64_t(num_sms) * 8));
    TraceScope trace("lora_dropout", stream);
    if (bf16) k_lora_dropout<true><<<static_cast<unsigned>(grid), kThreads, 0, stream>>>(in, n, drop, out);
    else k_lora_dropout<false><<<static_cast<unsigned>(grid), kThreads, 0, stream>>>(in, n, drop, out);
    return cudaGetLastError();
}

}  // namespace nf4lora
