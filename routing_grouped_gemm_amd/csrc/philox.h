// The counter-based generator behind dropout: Philox 4x32 with ten rounds
// (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3",
// 2011), one 128-bit result for each eight elements of a tensor.
//
// Sixteen bits an element: an element's decision costs an eighth of a
// generator call.  A call is twenty 32 x 32 -> 64 bit products, which issue at a
// quarter of the rate of an addition, so with 32 bits an element the generator
// and not the memory would bound a dropout of bf16 rows.  The probability is
// then a multiple of 2^-16; the kept elements' factor is made from that
// multiple, so the mean is right.
#pragma once

#include "moe_internal.h"

namespace moe {

struct PhiloxKey {
    uint32_t k0, k1, c2, c3;   // seed, and the step as the counter's upper half
};

__device__ __forceinline__ PhiloxKey philox_key(const uint64_t* rng)
{
    const uint64_t seed = rng[0], step = rng[1];
    return {(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)step, (uint32_t)(step >> 32)};
}

__device__ __forceinline__ uint4 philox(PhiloxKey k, uint64_t block)
{
    uint32_t x0 = (uint32_t)block, x1 = (uint32_t)(block >> 32), x2 = k.c2, x3 = k.c3;
    uint32_t k0 = k.k0, k1 = k.k1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)x0 * 0xD2511F53u, b = (uint64_t)x2 * 0xCD9E8D57u;
        x0 = (uint32_t)(b >> 32) ^ x1 ^ k0;
        x2 = (uint32_t)(a >> 32) ^ x3 ^ k1;
        x1 = (uint32_t)b;
        x3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(x0, x1, x2, x3);
}

// the two elements that one result word decides
__device__ __forceinline__ bool keep_lo(uint32_t r, uint32_t thr) { return (r & 0xffffu) >= thr; }
__device__ __forceinline__ bool keep_hi(uint32_t r, uint32_t thr) { return (r >> 16) >= thr; }

// The decisions of four blocks as bits: element j of block i is dropped where bit 31 - (8 i + j) is set.
// push_bits() takes the blocks in order.
__device__ __forceinline__ uint32_t push_bits(uint32_t bits, uint4 r, uint32_t thr)
{
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        // the sign of the difference shifted in
        bits = __builtin_amdgcn_alignbit(bits, (w[q] & 0xffffu) - thr, 31);
        bits = __builtin_amdgcn_alignbit(bits, (w[q] >> 16) - thr, 31);
    }
    return bits;
}

// eight bf16 with the dropped ones of block i zero
__device__ __forceinline__ uint4 mask_vec(uint4 v, uint32_t bits, int i)
{
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t lo = (uint32_t)((int32_t)(bits << (8 * i + 2 * q)) >> 31);
        const uint32_t hi = (uint32_t)((int32_t)(bits << (8 * i + 2 * q + 1)) >> 31);
        w[q] &= ~((lo & 0xffffu) | (hi & 0xffff0000u));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace moe
