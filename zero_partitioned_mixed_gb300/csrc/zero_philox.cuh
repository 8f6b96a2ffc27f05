// Dropout's numbers: 16 bits an element from Philox4x32-10 (Salmon, Moraes,
// Dror, Shaw: "Parallel random numbers: as easy as 1, 2, 3", SC 2011), a
// generator without state, so that no mask is stored: the backward pass asks
// for the same numbers again.
//
// The key is the seed; the counter's low 64 bits are the number of a group of
// 8 consecutive columns, row * ceil(cols / 8) + col / 8, its high 64 bits the
// stream (the caller's offset, plus a word of device memory where a captured
// graph is to get other numbers each time it runs).  Of the 4 words, the low
// half of the first belongs to the first column, its high half to the second.
//
// 16 bits and not 32: 20 wide products serve 8 elements instead of 4, and
// with 32 bits the products alone would take longer than HBM for the data.
// The share that is dropped is then a multiple of 2^-16, and the factor of
// what is kept the inverse of just that share's complement: the mean stays
// as it was.
#pragma once

#include "zero_host.h"
#include "zero_rows.cuh"

namespace zg {
namespace {

struct DropArgs {
    uint32_t key0[10], key1[10];   // the rounds' keys
    uint64_t offset;
    const uint64_t* step;          // or NULL
    uint32_t below;                // an element is dropped when its 16 bits, as the high half of a word, lie below
    float factor;                  // of what is kept
};

// What the kernels take of the caller's dropout; `below` 0 where nothing is dropped.
inline int drop_args(DropArgs& a, const zero_dropout_t* d) {
    a = DropArgs{};
    a.factor = 1.0f;
    if (!d) return ZERO_OK;
    if (!(d->p >= 0.0 && d->p < 1.0)) return refuse(ZERO_EINVAL, "p must lie in [0, 1)");
    if (d->step && !aligned(d->step, 8)) return refuse(ZERO_EINVAL, "step is not 8-byte aligned");
    uint32_t drop = static_cast<uint32_t>(d->p * 65536.0 + 0.5);
    if (drop > 65535u) drop = 65535u;
    uint32_t k0 = static_cast<uint32_t>(d->seed), k1 = static_cast<uint32_t>(d->seed >> 32);
    for (int i = 0; i < 10; ++i, k0 += 0x9E3779B9u, k1 += 0xBB67AE85u) {
        a.key0[i] = k0;
        a.key1[i] = k1;
    }
    a.offset = d->offset;
    a.step = d->step;
    a.below = drop << 16;
    a.factor = static_cast<float>(65536.0 / (65536.0 - drop));
    return ZERO_OK;
}

__device__ __forceinline__ uint64_t drop_stream(const DropArgs& a) { return a.offset + (a.step ? *a.step : 0ull); }

__device__ __forceinline__ uint4 philox(const DropArgs& a, uint64_t group, uint64_t stream) {
    uint32_t x0 = static_cast<uint32_t>(group), x1 = static_cast<uint32_t>(group >> 32);
    uint32_t x2 = static_cast<uint32_t>(stream), x3 = static_cast<uint32_t>(stream >> 32);
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p = static_cast<uint64_t>(0xD2511F53u) * x0, q = static_cast<uint64_t>(0xCD9E8D57u) * x2;
        x0 = static_cast<uint32_t>(q >> 32) ^ x1 ^ a.key0[i];
        x1 = static_cast<uint32_t>(q);
        x2 = static_cast<uint32_t>(p >> 32) ^ x3 ^ a.key1[i];
        x3 = static_cast<uint32_t>(p);
    }
    return make_uint4(x0, x1, x2, x3);
}

// The dropout of a lane's eight values: a kept one times the factor, rounded
// once; a dropped one is 0, whatever it was.  By all lanes of a warp together;
// group: the lane's, of the 32 groups of a warp's 256 columns.  Where the lane
// has other columns than its group's (column_of), the groups' decisions are
// handed round.
template <bool ALIGNED>
__device__ __forceinline__ void drop_eight(const DropArgs& a, uint64_t group, uint64_t stream, float (&v)[8]) {
    const uint4 w = philox(a, group, stream);
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
    mul8(v, a.factor);
    if constexpr (ALIGNED) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = (r[i] << 16) < a.below ? 0.0f : v[2 * i];
            v[2 * i + 1] = r[i] < a.below ? 0.0f : v[2 * i + 1];
        }
    } else {
        uint32_t dropped = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            dropped |= (r[i] << 16) < a.below ? 1u << (2 * i) : 0u;
            dropped |= r[i] < a.below ? 2u << (2 * i) : 0u;
        }
        const uint32_t lane = threadIdx.x & 31, bit = 1u << (lane & 7);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = __shfl_sync(0xFFFFFFFFu, dropped, 4 * e + (lane >> 3)) & bit ? 0.0f : v[e];
    }
}

}  // namespace
}  // namespace zg
