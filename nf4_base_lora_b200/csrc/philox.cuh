// Counter-based keep decisions for dropout: nothing about the mask is stored,
// the forward and the backward generate it again where they need it.
//
// Generator: Philox4x32 with 7 rounds (Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", SC 2011: seven rounds are the
// fewest that pass every test of their battery; ten leave a margin that a keep
// decision does not need, and each round costs two wide multiplies).  Elements
// are taken in groups of eight consecutive ones: the counter of a group is
// (group low, group high, offset low, offset high), the key (seed low, seed
// high), and the four output words give each element 16 bits, of which the low
// 15, u, decide: kept iff u >= threshold = round(p 2^15).  15 bits and not 16
// because a sum then tells all pairs apart without a carry between halves:
// (u & 0x7FFF) + (0x8000 - threshold) has bit 15 set iff u >= threshold.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace nf4lora {

// threshold 0: nothing is dropped, rng is not read.  gain = 2^15 / (2^15 - threshold).
struct DropArgs {
    const int64_t* rng;  // device: {seed, offset}
    uint32_t threshold;
    float gain;
};

constexpr int kPhiloxRounds = 7;

struct KeepGen {
    uint32_t k0[kPhiloxRounds], k1[kPhiloxRounds];  // round keys
    uint32_t c2, c3;                                // the offset
    uint32_t add;                                   // 0x8000 - threshold in both halves

    __device__ __forceinline__ void init(const DropArgs& d) {
        const uint64_t seed = static_cast<uint64_t>(__ldcg(reinterpret_cast<const long long*>(d.rng)));
        const uint64_t off = static_cast<uint64_t>(__ldcg(reinterpret_cast<const long long*>(d.rng) + 1));
#pragma unroll
        for (int i = 0; i < kPhiloxRounds; ++i) {
            k0[i] = static_cast<uint32_t>(seed) + static_cast<uint32_t>(i) * 0x9E3779B9u;
            k1[i] = static_cast<uint32_t>(seed >> 32) + static_cast<uint32_t>(i) * 0xBB67AE85u;
        }
        c2 = static_cast<uint32_t>(off);
        c3 = static_cast<uint32_t>(off >> 32);
        add = (0x8000u - d.threshold) * 0x10001u;
    }

    // Bits 15 and 31 of f[i]: elements 2i and 2i + 1 of the group are kept.
    __device__ __forceinline__ void flags(uint64_t group, uint32_t (&f)[4]) const {
        uint32_t a = static_cast<uint32_t>(group), b = static_cast<uint32_t>(group >> 32), c = c2, d = c3;
#pragma unroll
        for (int i = 0; i < kPhiloxRounds; ++i) {
            const uint64_t pa = static_cast<uint64_t>(a) * 0xD2511F53u, pc = static_cast<uint64_t>(c) * 0xCD9E8D57u;
            a = static_cast<uint32_t>(pc >> 32) ^ b ^ k0[i];
            b = static_cast<uint32_t>(pc);
            c = static_cast<uint32_t>(pa >> 32) ^ d ^ k1[i];
            d = static_cast<uint32_t>(pa);
        }
        f[0] = (a & 0x7FFF7FFFu) + add;
        f[1] = (b & 0x7FFF7FFFu) + add;
        f[2] = (c & 0x7FFF7FFFu) + add;
        f[3] = (d & 0x7FFF7FFFu) + add;
    }

    // 0xFFFF in each half of m[i] whose element is kept, else 0 (the sign of
    // bytes 1 and 3 replicated over their halves).
    __device__ __forceinline__ void masks(uint64_t group, uint32_t (&m)[4]) const {
        flags(group, m);
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("prmt.b32 %0, %1, 0, 0xBB99;" : "=r"(m[i]) : "r"(m[i]));
    }
};

}  // namespace nf4lora
