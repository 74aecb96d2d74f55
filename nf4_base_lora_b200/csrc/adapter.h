// Internal interface between the C ABI (api.cu) and the adapter-dropout and
// grouped-expert operators (dropout.cu, grouped.cu).  Host-side, C++ linkage.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "philox.cuh"

namespace nf4lora {

// Value of the device status word (1: a bounded wait ran out): a group offset
// was negative, beyond M or smaller than the one before it.
constexpr int kStatusOffsets = 2;

cudaError_t launch_lora_dropout(const void* in, int64_t n, bool bf16, const DropArgs& drop, void* out, int num_sms,
                                cudaStream_t stream);

// E stacked encoded weights [E N, K], the rows offsets[e] .. offsets[e + 1] - 1
// of X [M, K] (device offsets) for expert e; offsets NULL: one weight, all rows.
struct GroupCtx {
    const uint8_t* codes;
    const int8_t* qscale;
    const float* scale2;
    const float* scale_mean;
    const float* absmax;  // fp32 block scales, or NULL
    int E;
    int64_t N, K, M;
    const int32_t* offsets;
    int r;
    float s;
    DropArgs drop;
    int num_sms;  // the split sizes assume this many (workspace sizes depend on the shape alone)
    cudaStream_t stream;
};

int64_t group_fwd_workspace_bytes(int64_t M, int E, int64_t N, int64_t K, int r, int num_sms);
int64_t group_bwd_workspace_bytes(int64_t M, int E, int64_t N, int64_t K, int r, int num_sms);

// The CUDA error of the last failed launch of the calling thread (then reset).
cudaError_t group_last_cuda_error();

// Return 0 on success, -1 if a tensor map could not be encoded, -2 if a launch failed.
int group_fwd(const GroupCtx& c, const uint16_t* A, const uint16_t* B, const uint16_t* X, uint16_t* Y, float* T_saved,
              uint8_t* ws);
int group_bwd(const GroupCtx& c, const uint16_t* A, const uint16_t* B, const uint16_t* X, const float* T_saved,
              const uint16_t* dY, uint16_t* dX, uint16_t* dA, uint16_t* dB, int accumulate, uint8_t* ws);

}  // namespace nf4lora
