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

// Rows of 16-bit matrices, eight values a lane: lane l of a warp has the row's
// group v of 8 consecutive values, lane l + 1 group v + 1.  ALIGNED: every row
// starts on 16 bytes and is whole eights.  Else a row that starts m values
// behind a 16-byte boundary is read as the two aligned pieces around a group
// and put together by shifts, and written in aligned pieces, each with the
// last m values of the lane before.
__device__ __noinline__ uint4 read_some(const unsigned short* at, int count) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < count) w[e >> 1] |= static_cast<uint32_t>(__ldcs(at + e)) << (16 * (e & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// Values `from` to `to` - 1 of eight.
__device__ __noinline__ void store_some(unsigned short* at, uint4 x, int from, int to) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e >= from && e < to) at[e] = static_cast<unsigned short>(w[e >> 1] >> (16 * (e & 1)));
}

// Zeros from value `valid` on: rare too.
__device__ __noinline__ uint4 without_tail(uint4 x, int valid) {
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
    clear_from(w, valid);
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void clear_tail(uint32_t (&w)[4], int valid) {
    const uint4 x = without_tail(make_uint4(w[0], w[1], w[2], w[3]), valid);
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
}

template <bool ALIGNED>
struct RowIn;
template <>
struct RowIn<true> {
    const uint4* first;
};
template <>
struct RowIn<false> {
    const uint4* first;          // the piece with the row's first value
    const unsigned short* row;
    uint32_t m;                  // values before that one in it; 8: pieces would leave the matrix, read value by value
};
// Row `row` of a rows x cols matrix.
template <bool ALIGNED>
__device__ __forceinline__ RowIn<ALIGNED> row_in(const unsigned short* base, uint64_t row, uint64_t ld, uint64_t rows, uint64_t cols) {
    const unsigned short* at = base + row * ld;
    if constexpr (ALIGNED) {
        return {reinterpret_cast<const uint4*>(at)};
    } else {
        const uintptr_t a = reinterpret_cast<uintptr_t>(at), first = a & ~static_cast<uintptr_t>(15);
        const uint32_t m = static_cast<uint32_t>(a - first) >> 1;
        const bool in = first >= reinterpret_cast<uintptr_t>(base) &&
                        first + 16 * ((m + cols + 7) / 8) <= reinterpret_cast<uintptr_t>(base + (rows - 1) * ld + cols);
        return {reinterpret_cast<const uint4*>(first), at, in ? m : 8u};
    }
}

// A read in two steps, so that a thread's loads are all in flight before the
// first one's values are looked at (putting them together takes branches).
template <bool ALIGNED>
struct Fetched {
    uint4 x;
};
template <>
struct Fetched<false> {
    uint4 x, y;
};
// Group v, `valid` (at most 8) of whose values are inside the row.
__device__ __forceinline__ void fetch8(const RowIn<true>& r, uint32_t v, int valid, Fetched<true>& f) {
    f.x = make_uint4(0u, 0u, 0u, 0u);
    if (valid > 0) f.x = __ldcs(r.first + v);
}
__device__ __forceinline__ void fetch8(const RowIn<false>& r, uint32_t v, int valid, Fetched<false>& f) {
    f.x = f.y = make_uint4(0u, 0u, 0u, 0u);
    if (r.m < 8u && valid > 0) f.x = r.first[v];
    if (r.m < 8u && valid > 8 - static_cast<int>(r.m)) f.y = r.first[v + 1];   // the next lane's first: the cache serves it
}
__device__ __forceinline__ void finish8(const RowIn<true>&, uint32_t, int, const Fetched<true>& f, uint32_t (&w)[4]) {
    w[0] = f.x.x; w[1] = f.x.y; w[2] = f.x.z; w[3] = f.x.w;
}
__device__ __forceinline__ void finish8(const RowIn<false>& r, uint32_t v, int valid, const Fetched<false>& f, uint32_t (&w)[4]) {
    if (r.m < 8u) {
        const uint32_t own[4] = {f.x.x, f.x.y, f.x.z, f.x.w}, next[4] = {f.y.x, f.y.y, f.y.z, f.y.w};
        shift_halves(own, next, r.m, w);
        if (valid < 8) clear_tail(w, valid);
    } else {
        const uint4 x = valid > 0 ? read_some(r.row + 8ull * v, valid) : make_uint4(0u, 0u, 0u, 0u);
        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    }
}
template <bool ALIGNED>
__device__ __forceinline__ void read8(const RowIn<ALIGNED>& r, uint32_t v, int valid, uint32_t (&w)[4]) {
    Fetched<ALIGNED> f;
    fetch8(r, v, valid, f);
    finish8(r, v, valid, f, w);
}

// The first m, and the last 8 - m, halves of an aligned piece; m in 1..7.
__device__ __forceinline__ void store_low(uint4* piece, const uint32_t (&q)[4], uint32_t m) {
    if (m & 4) *reinterpret_cast<uint2*>(piece) = make_uint2(q[0], q[1]);
    if (m & 2) reinterpret_cast<uint32_t*>(piece)[m & 4 ? 2 : 0] = m & 4 ? q[2] : q[0];
    if (m & 1) reinterpret_cast<unsigned short*>(piece)[m - 1] =
        static_cast<unsigned short>(m == 1 ? q[0] : m == 3 ? q[1] : m == 5 ? q[2] : q[3]);
}
__device__ __forceinline__ void store_high(uint4* piece, const uint32_t (&q)[4], uint32_t m) {
    const uint32_t k = (m + 1) >> 1;   // whole words from the k-th on
    if (m & 1) reinterpret_cast<unsigned short*>(piece)[m] =
        static_cast<unsigned short>((m == 1 ? q[0] : m == 3 ? q[1] : m == 5 ? q[2] : q[3]) >> 16);
    if (k & 1) reinterpret_cast<uint32_t*>(piece)[k] = k == 1 ? q[1] : q[3];
    if (k <= 2) reinterpret_cast<uint2*>(piece)[1] = make_uint2(q[2], q[3]);
}
// A row's groups written by all lanes of a warp together, 32 consecutive ones
// at a time and these one after the other (put), and at the end what is left
// between this warp and the next (finish).  Not ALIGNED: a lane writes the
// aligned piece with the last values of the lane before it, lane 0 with those
// that lane 31 had the last time; the piece between two warps is written by
// lane 0 of either; what ends the row is written value by value.
template <bool ALIGNED>
struct RowOut;
template <>
struct RowOut<true> {
    uint4* row;
    __device__ __forceinline__ explicit RowOut(unsigned short* at) : row(reinterpret_cast<uint4*>(at)) {}
    // `next`: how many values of group v + 1 are inside the row
    template <bool FIRST, bool LAST>
    __device__ __forceinline__ void put(uint32_t v, int valid, int, const uint32_t (&w)[4]) {
        if (valid > 0) __stcs(row + v, make_uint4(w[0], w[1], w[2], w[3]));
    }
};
template <>
struct RowOut<false> {
    unsigned short* row;
    uint32_t m;          // values between the row's first piece's start and the row: the same in all lanes
    uint32_t carry[4];   // lane 0: what lane 31 had
    __device__ __forceinline__ explicit RowOut(unsigned short* at)
        : row(at), m(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(at) >> 1) & 7u), carry{0u, 0u, 0u, 0u} {}
    template <bool FIRST, bool LAST>
    __device__ __forceinline__ void put(uint32_t v, int valid, int next, const uint32_t (&w)[4]) {
        const uint32_t lane = threadIdx.x & 31;
        unsigned short* at = row + 8ull * v;
        const int own = 8 - static_cast<int>(m);   // values up to the boundary
        int from = 0, to = 0;                      // values to be written by themselves
        if (m == 0u) {
            if (valid == 8) *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
            else to = valid;
        } else {
            uint32_t before[4], q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t round = __shfl_sync(0xFFFFFFFFu, w[i], (lane + 31) & 31);
                before[i] = lane == 0 ? carry[i] : round;
                carry[i] = round;
            }
            shift_halves(before, w, static_cast<uint32_t>(own), q);
            uint4* piece = reinterpret_cast<uint4*>(at - m);
            if (valid >= own) {
                if (FIRST && lane == 0) store_high(piece, q, m);
                else *piece = make_uint4(q[0], q[1], q[2], q[3]);
            }
            if (valid < own) to = valid;
            else if (valid > own && (LAST && lane == 31 ? valid < 8 : next < own)) from = own, to = valid;
            if (LAST && __shfl_sync(0xFFFFFFFFu, valid, 31) == 8 && lane == 0) {
                const uint32_t none[4] = {0u, 0u, 0u, 0u};
                shift_halves(carry, none, static_cast<uint32_t>(own), q);
                store_low(piece + 32, q, m);
            }
        }
        if (from < to) store_some(at, make_uint4(w[0], w[1], w[2], w[3]), from, to);
    }
};
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
