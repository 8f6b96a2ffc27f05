// Microscaled floats (the OCP MX formats) as the kernels here make and read
// them: blocks of 32 consecutive values of a row with one power-of-two scale,
// elements of 4 bits (e2m1) or 8 (e4m3).
//
// With E the exponent of the block's largest magnitude, its scale is
// 2^(E - T), T the largest exponent of the element type (2 and 8), stored as
// a byte with a bias of 127 and never below 2^-127; a value's code is
// x / scale rounded to the nearest value of the element type (0, 0.5, 1, 1.5,
// 2, 3, 4, 6, or e4m3's up to 448), ties to the even code, larger ones
// becoming the largest.  The division is a multiplication by a power of two
// and exact.  A block that holds an infinity or a NaN gets the scale 255,
// which stands for NaN, and codes of 0.
//
// Layout.  Codes: row by row, 4-bit ones two a byte, the even one low, every
// row filled with zeros to whole blocks.  Scales: tiles of 128 rows x 4
// blocks, 512 bytes each, row-major over the matrix; in a tile, byte
// 16 (r mod 32) + 4 (r / 32) + b.  That is what the tensor cores take: a tile
// is copied into tensor memory as it stands.  The tiles' unused bytes are 0.
#pragma once

#include <cstdint>
#include <type_traits>

#include "zero_rows.cuh"

namespace zg {
namespace {

constexpr int kMxBlock = ZERO_MX_BLOCK;

template <int BITS>
struct MxElement {
    static_assert(BITS == 4 || BITS == 8, "e2m1 or e4m3");
    static constexpr uint32_t kTop = BITS == 4 ? 2 : 8;              // the largest exponent
    using Eight = std::conditional_t<BITS == 4, uint32_t, uint2>;    // 8 codes as they are stored, the first one lowest
};

__host__ __device__ __forceinline__ uint64_t scale_at(uint64_t row, uint64_t block, uint64_t tiles_k) {
    return ((row >> 7) * tiles_k + (block >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (block & 3);
}

// The scale byte of a block from the bits of its largest magnitude.
template <int BITS>
__device__ __forceinline__ uint32_t scale_byte(float top) {
    const uint32_t e = __float_as_uint(top) >> 23;   // 255: infinity or NaN
    return e == 255u ? 255u : e > MxElement<BITS>::kTop ? e - MxElement<BITS>::kTop : 0u;
}
// 1 / scale; 0 for a NaN block, whose codes are 0.
__device__ __forceinline__ float scale_inverse(uint32_t byte) {
    return byte == 255u ? 0.0f : __uint_as_float((254u - byte) << 23);
}
// What a scale byte stands for: 2^(byte - 127), the smallest a subnormal number.
__device__ __forceinline__ float scale_value(uint32_t byte) {
    return byte == 255u ? NAN : __uint_as_float(byte == 0u ? 0x00400000u : byte << 23);
}

// 8 values as codes, the first in the lowest bits.
__device__ __forceinline__ void codes8(const float (&x)[8], uint32_t& r) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
}
__device__ __forceinline__ uint32_t codes4_e4m3(float x0, float x1, float x2, float x3) {
    uint32_t r;
    asm("{\n\t.reg .b16 a, b;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
        "mov.b32 %0, {a, b};\n\t}"
        : "=r"(r)
        : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
    return r;
}
__device__ __forceinline__ void codes8(const float (&x)[8], uint2& r) {
    r.x = codes4_e4m3(x[0], x[1], x[2], x[3]);
    r.y = codes4_e4m3(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void no_codes(uint32_t& r) { r = 0u; }
__device__ __forceinline__ void no_codes(uint2& r) { r = make_uint2(0u, 0u); }

// Codes 2 e and 2 e + 1 of eight, as fp32 (both types' values are values of fp16).
__device__ __forceinline__ void decode2(uint32_t eight, int e, float& lo, float& hi) {
    uint32_t h;
    asm("{\n\t.reg .b8 b, x, y, z;\n\tmov.b32 {b, x, y, z}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}"
        : "=r"(h)
        : "r"(eight >> (8 * e)));
    widen2<kFp16>(h, lo, hi);
}
__device__ __forceinline__ void decode2(uint2 eight, int e, float& lo, float& hi) {
    uint32_t h;
    const uint32_t w = (e & 2 ? eight.y : eight.x) >> (16 * (e & 1));
    asm("{\n\t.reg .b16 b, x;\n\tmov.b32 {b, x}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}" : "=r"(h) : "r"(w));
    widen2<kFp16>(h, lo, hi);
}
// The 8 codes that begin m (1..7) codes before `word` does: the last m of the
// word before it, then its own.
__device__ __forceinline__ uint32_t codes_before(uint32_t before, uint32_t word, int m) {
    return __funnelshift_r(before, word, 4 * (8 - m));
}
__device__ __forceinline__ uint2 codes_before(uint2 before, uint2 word, int m) {
    const uint64_t b = before.x | static_cast<uint64_t>(before.y) << 32, w = word.x | static_cast<uint64_t>(word.y) << 32;
    const uint64_t r = (b >> (8 * (8 - m))) | (w << (8 * m));
    return make_uint2(static_cast<uint32_t>(r), static_cast<uint32_t>(r >> 32));
}

}  // namespace
}  // namespace zg
