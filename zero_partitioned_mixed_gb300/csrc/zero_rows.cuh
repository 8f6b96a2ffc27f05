// A warp's reads of 256 consecutive 16-bit values of a row-major matrix whose
// rows may start anywhere: 8 values a lane, as the aligned 16-byte pieces that
// cover them, whatever the row's alignment.  Only pieces that would leave the
// matrix are read value by value, so nothing outside of it is touched.
#pragma once

#include "zero_device.cuh"

namespace zg {
namespace {

// Halves m to m + 7 of the 16 halves lo, hi; m in 1..7 and the same in all
// lanes.
__device__ __forceinline__ void shift_halves(const uint32_t (&lo)[4], const uint32_t (&hi)[4], uint32_t m,
                                             uint32_t (&out)[4]) {
    uint32_t w[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    if (m & 4) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (m & 2) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = __funnelshift_r(w[i], w[i + 1], 16 * (m & 1));
}

// The aligned piece whose first value is `at` (which may lie before the
// matrix), values outside [0, total) as 0.
__device__ __forceinline__ void load_piece(const unsigned short* base, int64_t at, int64_t total, uint32_t (&w)[4]) {
    if (at >= 0 && at + 8 <= total) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(base + at));
        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t a = at + 2 * i;
            const uint32_t lo = a >= 0 && a < total ? __ldg(base + a) : 0u;
            const uint32_t hi = a + 1 >= 0 && a + 1 < total ? __ldg(base + a + 1) : 0u;
            w[i] = lo | hi << 16;
        }
    }
}

// This lane's 8 values (packed pairs) from value `at` of the matrix on; lanes
// of a warp take consecutive eights.  `total`: values from `base` to the
// matrix's end.  Values past a row's end are the caller's to ignore.
__device__ __forceinline__ void load8(const unsigned short* base, int64_t at, int64_t total, uint32_t (&w)[4]) {
    const uint32_t m = static_cast<uint32_t>((reinterpret_cast<uintptr_t>(base) >> 1) + static_cast<uint64_t>(at)) & 7u;
    if (m == 0) {
        load_piece(base, at, total, w);
        return;
    }
    uint32_t own[4], next[4];   // two pieces, the second one the next lane's first: the cache serves it
    if (at >= static_cast<int64_t>(m) && at + 16 <= total) {
        const uint4* from = reinterpret_cast<const uint4*>(base + at - m);
        const uint4 x = __ldg(from), y = __ldg(from + 1);
        own[0] = x.x; own[1] = x.y; own[2] = x.z; own[3] = x.w;
        next[0] = y.x; next[1] = y.y; next[2] = y.z; next[3] = y.w;
    } else {
        load_piece(base, at - m, total, own);
        load_piece(base, at - m + 8, total, next);
    }
    shift_halves(own, next, m, w);
}

// A lane's values left of a row's `cols` from column c on, within +-8.
__device__ __forceinline__ int values_left(uint64_t cols, uint64_t c) {
    const int64_t left = static_cast<int64_t>(cols) - static_cast<int64_t>(c);
    return left > 8 ? 8 : left < -8 ? -8 : static_cast<int>(left);
}
// Zeros in place of the values from `valid` on.
__device__ __forceinline__ void clear_from(uint32_t (&w)[4], int valid) {
    if (valid >= 8) return;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = valid >= 2 * i + 2 ? w[i] : valid == 2 * i + 1 ? w[i] & 0xFFFFu : 0u;
}
// The largest magnitude of 8 values as a 16-bit pattern: patterns are ordered
// like magnitudes in both formats, infinity and NaN above every number.
__device__ __forceinline__ uint32_t top_pattern(const uint32_t (&w)[4]) {
    const uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                                __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
    return max(m & 0xFFFFu, m >> 16);
}
// Both values of a word.
template <int DT>
__device__ __forceinline__ void widen2(uint32_t w, float& lo, float& hi) {
    if (DT == kBf16) {
        lo = __uint_as_float(w << 16);
        hi = __uint_as_float(w & 0xFFFF0000u);
    } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        lo = f.x;
        hi = f.y;
    }
}
// Two fp32 values as packed 16-bit ones, the first in the low half.
template <int DT>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
    uint32_t r;
    if (DT == kBf16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two products, each rounded once.
__device__ __forceinline__ void mul2(float& a, float& b, float by) {
    unsigned long long x, y;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b));
    asm("mov.b64 %0, {%1, %1};" : "=l"(y) : "f"(by));
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(x) : "l"(y));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
// Eight at a time, in pairs: one instruction for two values, each rounded as
// by itself.
__device__ __forceinline__ unsigned long long pair(float a, float b) {
    unsigned long long x;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b));
    return x;
}
__device__ __forceinline__ void unpair(unsigned long long x, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ void mul8(float (&a)[8], float by) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) mul2(a[e], a[e + 1], by);
}
__device__ __forceinline__ void mul8(float (&a)[8], const float (&b)[8]) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        unsigned long long x;
        asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(x) : "l"(pair(a[e], a[e + 1])), "l"(pair(b[e], b[e + 1])));
        unpair(x, a[e], a[e + 1]);
    }
}
__device__ __forceinline__ void add8(float (&a)[8], const float (&b)[8]) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        unsigned long long x;
        asm("add.rn.f32x2 %0, %1, %2;" : "=l"(x) : "l"(pair(a[e], a[e + 1])), "l"(pair(b[e], b[e + 1])));
        unpair(x, a[e], a[e + 1]);
    }
}
// a b + c, rounded once.
__device__ __forceinline__ void fma8(const float (&a)[8], const float (&b)[8], float (&c)[8]) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        unsigned long long x;
        asm("fma.rn.f32x2 %0, %1, %2, %3;"
            : "=l"(x)
            : "l"(pair(a[e], a[e + 1])), "l"(pair(b[e], b[e + 1])), "l"(pair(c[e], c[e + 1])));
        unpair(x, c[e], c[e + 1]);
    }
}
// The sum over the eight of a b, into two running sums.
__device__ __forceinline__ void dot8(const float (&a)[8], const float (&b)[8], float (&s)[2]) {
    unsigned long long x = pair(s[0], s[1]);
#pragma unroll
    for (int e = 0; e < 8; e += 2)
        asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(x) : "l"(pair(a[e], a[e + 1])), "l"(pair(b[e], b[e + 1])));
    unpair(x, s[0], s[1]);
}

// 256 columns of a row of 16-bit values at a time, by a warp, eight a lane.
// ALIGNED, where every row starts on 16 bytes and is whole eights: lane l has
// columns 8 l to 8 l + 7.  Else it has columns l, l + 32, ..., l + 224, so that
// every access of the warp is 64 neighbouring bytes wherever the row starts,
// nothing has to be shifted together, and nothing beside the row is touched.
// (Aligned 16-byte pieces put together by shifts, the lanes at a warp's ends
// writing theirs in parts, took 89 us for 4001 x 5003 bf16 through the norm's
// backward pass against 69 so, 15.8 against 11.4 for 2047 x 1003 fp16 and 4.9
// against 3.7 through dropout, 25 against 13 for looking up 8001 x 2001.)
template <bool ALIGNED>
__device__ __forceinline__ uint32_t column_of(int e) {
    const uint32_t lane = threadIdx.x & 31;
    return ALIGNED ? 8 * lane + e : 32 * e + lane;
}
template <bool ALIGNED>
struct Loaded;
template <>
struct Loaded<true> {
    uint4 x;
};
template <>
struct Loaded<false> {
    unsigned short x[8];
};
// at: the first of the 256 columns, `left` of which (any number) are inside
// the row; zeros for the others.
__device__ __forceinline__ void load_eight(const unsigned short* at, int left, Loaded<true>& r) {
    r.x = make_uint4(0u, 0u, 0u, 0u);
    if (static_cast<int>(column_of<true>(0)) < left) r.x = __ldcs(reinterpret_cast<const uint4*>(at) + (threadIdx.x & 31));
}
__device__ __forceinline__ void load_eight(const unsigned short* at, int left, Loaded<false>& r) {
    at += threadIdx.x & 31;
    if (left >= 256) {   // the same in all lanes
#pragma unroll
        for (int e = 0; e < 8; ++e) r.x[e] = __ldcs(at + 32 * e);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) r.x[e] = static_cast<int>(column_of<false>(e)) < left ? __ldcs(at + 32 * e) : 0;
    }
}
template <int DT>
__device__ __forceinline__ void widen_eight(const Loaded<true>& r, float (&v)[8]) {
    widen2<DT>(r.x.x, v[0], v[1]);
    widen2<DT>(r.x.y, v[2], v[3]);
    widen2<DT>(r.x.z, v[4], v[5]);
    widen2<DT>(r.x.w, v[6], v[7]);
}
template <int DT>
__device__ __forceinline__ void widen_eight(const Loaded<false>& r, float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = widen<DT>(r.x[e]);
}
// q: the eight in pairs, the first one low.
template <bool ALIGNED>
__device__ __forceinline__ void store_eight(unsigned short* at, int left, const uint32_t (&q)[4]) {
    if constexpr (ALIGNED) {
        if (static_cast<int>(column_of<true>(0)) < left)
            __stcs(reinterpret_cast<uint4*>(at) + (threadIdx.x & 31), make_uint4(q[0], q[1], q[2], q[3]));
    } else {
        at += threadIdx.x & 31;
        if (left >= 256) {   // the same in all lanes
#pragma unroll
            for (int e = 0; e < 8; ++e) at[32 * e] = static_cast<unsigned short>(q[e >> 1] >> (16 * (e & 1)));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (static_cast<int>(column_of<false>(e)) < left)
                    at[32 * e] = static_cast<unsigned short>(q[e >> 1] >> (16 * (e & 1)));
        }
    }
}
// How many of the 256 columns from `first` on are inside a row of `cols`.
__device__ __forceinline__ int columns_left(uint64_t cols, uint64_t first) {
    const int64_t left = static_cast<int64_t>(cols) - static_cast<int64_t>(first);
    return left > 256 ? 256 : left < 0 ? 0 : static_cast<int>(left);
}
template <int DT>
__device__ __forceinline__ void widen8(const uint32_t (&w)[4], float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) widen2<DT>(w[i], v[2 * i], v[2 * i + 1]);
}
template <int DT>
__device__ __forceinline__ void narrow8(const float (&v)[8], uint32_t (&w)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = narrow2<DT>(v[2 * i], v[2 * i + 1]);
}

}  // namespace
}  // namespace zg
