// Microscaled 4-bit floats (the OCP MX format with e2m1 elements): quantising
// a matrix along its rows or its columns, reading it back, and the product of
// two such matrices on the block-scaled tensor cores.
//
// A block is 32 consecutive values of a row.  With E the exponent of the
// block's largest magnitude, its scale is 2^(E - 2) (2 is e2m1's largest
// exponent), stored as a byte with a bias of 127 and never below 2^-127; a
// value's code is x / scale rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3,
// 4, 6 (ties to the even code), larger ones becoming 6.  The division is a
// multiplication by a power of two and exact.  A block that holds an
// infinity or a NaN gets the scale 255, which stands for NaN, and codes of 0.
//
// Layout.  Codes: row by row, two a byte, the even one low, every row filled
// with zeros to whole blocks.  Scales: tiles of 128 rows x 4 blocks, 512
// bytes each, row-major over the matrix; in a tile, byte 16 (r mod 32) +
// 4 (r / 32) + b.  That is what the tensor cores take: a tile is copied into
// tensor memory as it stands.  The tiles' unused bytes are 0.

#include <atomic>
#include <cstdint>
#include <string>

#include <nvtx3/nvToolsExt.h>

#include "zero_gb300.h"
#include "zero_rows.cuh"
#include "zero_tc.cuh"

namespace zg {
namespace {

constexpr int kMxBlock = ZERO_MX_BLOCK;

struct MxArgs {
    const void* src;
    void* dst;
    uint8_t* codes;
    uint8_t* scales;
    uint64_t rows, cols, ld;   // of the 16-bit matrix
    uint64_t pitch;            // bytes of a row of codes
    uint64_t tiles_k;          // scale tiles along a row of codes
};

__device__ __forceinline__ uint64_t scale_at(uint64_t row, uint64_t block, uint64_t tiles_k) {
    return ((row >> 7) * tiles_k + (block >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (block & 3);
}

// The scale byte of a block from the bits of its largest magnitude.
__device__ __forceinline__ uint32_t scale_byte(float top) {
    const uint32_t e = __float_as_uint(top) >> 23;   // 255: infinity or NaN
    return e == 255u ? 255u : e > 2u ? e - 2u : 0u;
}
// 1 / scale; 0 for a NaN block, whose codes are 0.
__device__ __forceinline__ float scale_inverse(uint32_t byte) {
    return byte == 255u ? 0.0f : __uint_as_float((254u - byte) << 23);
}
// 8 values as codes, the first in the lowest 4 bits.
__device__ __forceinline__ uint32_t codes8(const float (&x)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

// The row kernels: a warp takes kMxRows rows by 256 columns, 8 a lane, all
// rows' loads in flight together.  They are bound by the instructions they
// issue as much as by HBM, so a piece that lies inside the matrix and starts
// on 16 bytes takes a path without any of the edges' cases (`INSIDE`): for
// 11008 x 4096 bf16 20 us to quantise (5.7 TB/s) and 23 us to read back (5.0
// TB/s) against 28 and 28 with one path for all.  Rows at odd strides: 8.2
// and 7.8 us for 2047 x 5003 against 7.4 and 5.9 for 2048 x 5000.
constexpr int kMxRows = 4;

template <int DT, bool INSIDE>
__device__ __forceinline__ void rows_piece(const MxArgs& a, uint64_t row0, uint64_t segment) {
    const int lane = threadIdx.x & 31;
    const uint64_t c = segment * 256 + 8 * lane;
    const unsigned short* src = static_cast<const unsigned short*>(a.src);
    const int valid = INSIDE ? 8 : values_left(a.cols, c);
    uint32_t raw[kMxRows][4];
    if (INSIDE) {
        const unsigned short* at = src + row0 * a.ld + c;
#pragma unroll
        for (int r = 0; r < kMxRows; ++r, at += a.ld) {
            const uint4 x = __ldcs(reinterpret_cast<const uint4*>(at));
            raw[r][0] = x.x; raw[r][1] = x.y; raw[r][2] = x.z; raw[r][3] = x.w;
        }
    } else {
        const int64_t total = static_cast<int64_t>((a.rows - 1) * a.ld + a.cols);
#pragma unroll
        for (int r = 0; r < kMxRows; ++r) {
            if (row0 + r < a.rows) {
                load8(src, static_cast<int64_t>((row0 + r) * a.ld + c), total, raw[r]);
                clear_from(raw[r], valid);
            } else {
                raw[r][0] = raw[r][1] = raw[r][2] = raw[r][3] = 0;
            }
        }
    }
    uint8_t* codes = a.codes + row0 * a.pitch + (c >> 1);
    // kMxRows rows of a scale tile follow each other at 16 bytes
    uint8_t* scales = a.scales + scale_at(row0, c >> 5, a.tiles_k);
#pragma unroll
    for (int r = 0; r < kMxRows; ++r, codes += a.pitch) {
        uint32_t top = top_pattern(raw[r]);
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));   // four lanes share a block
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        const uint32_t byte = scale_byte(widen<DT>(top));
        const float inv = scale_inverse(byte);
        float v[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            widen2<DT>(raw[r][e], v[2 * e], v[2 * e + 1]);
            mul2(v[2 * e], v[2 * e + 1], inv);
        }
        const uint32_t q = byte == 255u ? 0u : codes8(v);
        if (INSIDE || (row0 + r < a.rows && (c >> 1) < a.pitch)) __stcs(reinterpret_cast<uint32_t*>(codes), q);
        // the four blocks of a scale tile's row in one word
        uint32_t word = byte | __shfl_down_sync(0xFFFFFFFFu, byte, 4) << 8;
        word |= __shfl_down_sync(0xFFFFFFFFu, word, 8) << 16;
        if ((lane & 15) == 0 && (INSIDE || (c >> 7) < a.tiles_k)) *reinterpret_cast<uint32_t*>(scales + 16 * r) = word;
    }
}

// Along the rows; those that only fill the last scale tiles are walked too,
// for their zeros.  ALIGNED: every row of the matrix starts on 16 bytes.
template <int DT, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) k_mx4_rows(const __grid_constant__ MxArgs a) {
    pdl_enter();
    const uint64_t row0 = (static_cast<uint64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * kMxRows;
    for (uint64_t segment = blockIdx.y; segment < (a.tiles_k + 1) / 2; segment += gridDim.y) {
        if (ALIGNED && row0 + kMxRows <= a.rows && (segment + 1) * 256 <= a.cols) rows_piece<DT, true>(a, row0, segment);
        else rows_piece<DT, false>(a, row0, segment);
    }
}

// Along the columns: the codes are those of the transpose.  A block takes
// 128 rows (a scale tile's four blocks) of 128 columns, a thread 32 values
// of two neighbouring columns; the codes go through shared memory so that a
// row of them leaves as 64 neighbouring bytes.  11008 x 4096: 18.6 us (6.1
// TB/s; one column a thread and codes straight from registers took 33).
template <int DT>
__global__ void __launch_bounds__(kThreads) k_mx4_columns(const __grid_constant__ MxArgs a) {
    pdl_enter();
    __shared__ __align__(16) uint4 s_codes[128][5];   // 5: neighbouring columns start in other banks
    __shared__ __align__(4) uint8_t s_scale[128][4];   // a row is read as one word
    const int lane = threadIdx.x & 31, b = (threadIdx.x >> 5) & 3;
    const int c = (threadIdx.x >> 7) * 64 + 2 * lane;
    const uint64_t col0 = static_cast<uint64_t>(blockIdx.x) * 128, row0 = static_cast<uint64_t>(blockIdx.y) * 128;
    const unsigned short* src = static_cast<const unsigned short*>(a.src) + (row0 + 32 * b) * a.ld + col0 + c;
    const bool inside = row0 + 128 <= a.rows && col0 + 128 <= a.cols;
    uint32_t raw[32];   // a row's two values each
    if (inside && (a.ld & 1) == 0 && (reinterpret_cast<uintptr_t>(a.src) & 3) == 0) {
#pragma unroll
        for (int e = 0; e < 32; ++e, src += a.ld) raw[e] = __ldg(reinterpret_cast<const uint32_t*>(src));
    } else if (inside) {
#pragma unroll
        for (int e = 0; e < 32; ++e, src += a.ld)
            raw[e] = static_cast<uint32_t>(__ldg(src)) | static_cast<uint32_t>(__ldg(src + 1)) << 16;
    } else {
        const uint64_t r0 = row0 + 32 * b;
        const int rows = r0 >= a.rows ? 0 : a.rows - r0 < 32 ? static_cast<int>(a.rows - r0) : 32;
        const int cols = col0 + c >= a.cols ? 0 : a.cols - col0 - c < 2 ? 1 : 2;
#pragma unroll
        for (int e = 0; e < 32; ++e, src += a.ld) {
            raw[e] = 0;
            if (e < rows && cols > 0) raw[e] = __ldg(src);
            if (e < rows && cols > 1) raw[e] |= static_cast<uint32_t>(__ldg(src + 1)) << 16;
        }
    }
    uint32_t tops = 0;
#pragma unroll
    for (int e = 0; e < 32; ++e) tops = __vmaxu2(tops, raw[e] & 0x7FFF7FFFu);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t byte = scale_byte(widen<DT>((tops >> (16 * h)) & 0xFFFFu));
        const float inv = scale_inverse(byte);
        uint32_t q[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                x[e] = widen<DT>((raw[8 * g + e] >> (16 * h)) & 0xFFFFu);
                x[e + 1] = widen<DT>((raw[8 * g + e + 1] >> (16 * h)) & 0xFFFFu);
                mul2(x[e], x[e + 1], inv);
            }
            q[g] = byte == 255u ? 0u : codes8(x);
        }
        s_codes[c + h][b] = make_uint4(q[0], q[1], q[2], q[3]);
        s_scale[c + h][b] = static_cast<uint8_t>(byte);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int cc = (threadIdx.x >> 2) + 64 * k, bb = threadIdx.x & 3;
        const uint64_t out = col0 + cc, at = (row0 + 32 * bb) / 2;
        if (out < a.cols && at < a.pitch) *reinterpret_cast<uint4*>(a.codes + out * a.pitch + at) = s_codes[cc][bb];
    }
    if (threadIdx.x < 128)   // the grid covers whole scale tiles
        *reinterpret_cast<uint32_t*>(a.scales + scale_at(col0 + threadIdx.x, 4 * static_cast<uint64_t>(blockIdx.y), a.tiles_k)) =
            *reinterpret_cast<const uint32_t*>(s_scale[threadIdx.x]);
}

// What a scale byte stands for: 2^(byte - 127), the smallest a subnormal number.
__device__ __forceinline__ float scale_value(uint32_t byte) {
    return byte == 255u ? NAN : __uint_as_float(byte == 0u ? 0x00400000u : byte << 23);
}
// Two codes (the low 8 bits of q) as fp32.
__device__ __forceinline__ void decode2(uint32_t q, float& lo, float& hi) {
    uint32_t h;
    asm("{\n\t.reg .b8 b, x, y, z;\n\tmov.b32 {b, x, y, z}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(h) : "r"(q));
    widen2<kFp16>(h, lo, hi);
}

// Rows that start on 16 bytes, 256 columns of them inside the matrix.
template <int DT>
__device__ __forceinline__ void values_inside(const MxArgs& a, uint64_t row0, uint64_t segment) {
    const uint64_t c = segment * 256 + 8 * (threadIdx.x & 31);
    const uint8_t* codes = a.codes + row0 * a.pitch + (c >> 1);
    const uint8_t* scales = a.scales + scale_at(row0, c >> 5, a.tiles_k);
    uint32_t q[kMxRows], byte[kMxRows];
#pragma unroll
    for (int r = 0; r < kMxRows; ++r, codes += a.pitch) {
        q[r] = __ldcs(reinterpret_cast<const uint32_t*>(codes));
        byte[r] = __ldg(scales + 16 * r);
    }
    unsigned short* dst = static_cast<unsigned short*>(a.dst) + row0 * a.ld + c;
#pragma unroll
    for (int r = 0; r < kMxRows; ++r, dst += a.ld) {
        const float scale = scale_value(byte[r]);
        uint32_t out[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float lo, hi;
            decode2(q[r] >> (8 * e), lo, hi);
            mul2(lo, hi, scale);
            out[e] = narrow2<DT>(lo, hi);
        }
        __stcs(reinterpret_cast<uint4*>(dst), make_uint4(out[0], out[1], out[2], out[3]));
    }
}

// Any rows and columns.  A lane writes an aligned piece of 16 bytes; where a
// row starts between two boundaries (not ALIGNED), the piece begins m values
// before a word of 8 codes does, and its first m values are the last ones of
// the word before, which may belong to another block.
template <int DT, bool ALIGNED>
__device__ __forceinline__ void values_any(const MxArgs& a, uint64_t row0, uint64_t segment) {
    const int64_t word = static_cast<int64_t>(segment) * 32 + (threadIdx.x & 31);   // along the row of codes
    const int64_t words = static_cast<int64_t>(a.pitch / 4), cols = static_cast<int64_t>(a.cols);
    // words past the row's ends stand for nothing that is written: any will do
    const int64_t here = min(word, words - 1), there = max(min(word - 1, words - 1), static_cast<int64_t>(0));
    const uint32_t* codes = reinterpret_cast<const uint32_t*>(a.codes + row0 * a.pitch);
    const uint8_t* scales = a.scales + scale_at(row0, here >> 2, a.tiles_k);
    const uint8_t* scales_before = a.scales + scale_at(row0, there >> 2, a.tiles_k);
    uint32_t q[kMxRows], before[kMxRows], byte[kMxRows], byte_before[kMxRows];
#pragma unroll
    for (int r = 0; r < kMxRows; ++r, codes += words) {
        if (row0 + r >= a.rows) break;
        q[r] = __ldg(codes + here);
        byte[r] = __ldg(scales + 16 * r);
        if (!ALIGNED) {
            before[r] = __ldg(codes + there);
            byte_before[r] = __ldg(scales_before + 16 * r);
        }
    }
    unsigned short* row = static_cast<unsigned short*>(a.dst) + row0 * a.ld;
#pragma unroll
    for (int r = 0; r < kMxRows; ++r, row += a.ld) {
        if (row0 + r >= a.rows) break;
        const int m = ALIGNED ? 0 : static_cast<int>((reinterpret_cast<uintptr_t>(row) >> 1) & 7);
        const float scale = scale_value(byte[r]), scale_before = ALIGNED ? 0.0f : scale_value(byte_before[r]);
        const uint32_t eight = m == 0 ? q[r] : __funnelshift_r(before[r], q[r], 4 * (8 - m));
        uint32_t out[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float lo, hi;
            decode2(eight >> (8 * e), lo, hi);
            lo = __fmul_rn(lo, 2 * e < m ? scale_before : scale);
            hi = __fmul_rn(hi, 2 * e + 1 < m ? scale_before : scale);
            out[e] = narrow2<DT>(lo, hi);
        }
        const int64_t c = 8 * word - m;
        if (c >= 0 && c + 8 <= cols) {
            __stcs(reinterpret_cast<uint4*>(row + c), make_uint4(out[0], out[1], out[2], out[3]));
        } else if (c < cols) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e >= 0 && c + e < cols) row[c + e] = static_cast<unsigned short>(out[e >> 1] >> (16 * (e & 1)));
        }
    }
}

// Codes and scales back to 16 bits.  ALIGNED: every row of the matrix starts
// on 16 bytes.
template <int DT, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) k_mx4_values(const __grid_constant__ MxArgs a) {
    pdl_enter();
    const uint64_t row0 = (static_cast<uint64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * kMxRows;
    if (row0 >= a.rows) return;
    // the pieces of a row that starts between boundaries may be one more than its words
    for (uint64_t segment = blockIdx.y; segment < (a.cols + (ALIGNED ? 0 : 7) + 255) / 256; segment += gridDim.y) {
        if (ALIGNED && row0 + kMxRows <= a.rows && (segment + 1) * 256 <= a.cols) values_inside<DT>(a, row0, segment);
        else values_any<DT, ALIGNED>(a, row0, segment);
    }
}

// ----------------------------------------------------------------- product
// out[m][n] = sum over k of A[m][k] B[n][k], fp32 accumulation.  A CTA
// computes 256 x 192 as two accumulators of 128 rows that share B's tile (MT
// 2), or 128 x 192 (MT 1).  A stage of 256 values of k is 60 KiB for 768
// cycles of products (43 for 384), so what an SM gets from L2 (some 50 bytes
// a cycle) bounds it and the larger tile is the better one as long as there
// are tiles for all SMs.  Two accumulators and four sets of scales fill
// tensor memory: one accumulator is written out while the other one's
// products run.  192 columns begin in the middle of a scale tile of 128 rows
// half of the time: two scale tiles cover them either way, and the product
// starts two columns further on in tensor memory.
struct MxProductArgs {
    uint32_t m, n, k;
    uint32_t tiles_m, tiles_n, total;
    uint32_t tiles_k;        // scale tiles along k
    void* out;
    uint64_t ld;
    int vec;                 // rows of out start on 16 bytes
    uint32_t hold;           // zero_debug_hold_matrix, or 0
};

constexpr int kMxN = 192, kMxK = 256;   // a stage's values of k are 128 bytes of a row
constexpr int kMxOutWarps = 8, kMxThreads = 64 + 32 * kMxOutWarps;
constexpr uint32_t kMxOut = 32 * 32 * 2;   // a warp's output buffer, two each
template <int MT>
struct MxTile {
    static constexpr uint32_t kRows = 128 * MT, kA = kRows * 128, kB = kMxN * 128, kScaleA = 1024 * MT, kScaleB = 2048;
    static constexpr uint32_t kStage = kA + kB + kScaleA + kScaleB;
    static constexpr int kStages = MT == 2 ? 3 : 4;   // at most the sets of scales: a set is free once its stage is
    static constexpr uint32_t kSet = 8 * MT + 16;     // columns of a set: 4 for 128 rows and 128 values of k
    static constexpr size_t kSmem = 1024 + kStages * kStage + kMxOutWarps * 2 * kMxOut;
    static_assert(2 * kMxN + 4 * kSet <= 512, "tensor memory");
    static_assert(kSmem >= kLeastTmemSmem, "see tmem_alloc");
};

// A scale tile (32 lines of 16 bytes in shared memory) into 4 columns of
// tensor memory, repeated in each quarter of the lanes.
__device__ __forceinline__ uint64_t scale_desc(uint32_t smem) {
    uint64_t d = static_cast<uint64_t>((smem & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(128u >> 4) << 32;   // 8 lines of 16 bytes
    d |= static_cast<uint64_t>(1) << 46;
    return d;
}
__device__ __forceinline__ void tc_copy_scales(uint32_t tmem, uint64_t d) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(d) : "memory");
}
__device__ __forceinline__ void mma_mx4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                        bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
}

// Tile t in bands of kBand tiles down, band after band: the tiles in flight
// at a time then share their operands in both directions.
constexpr uint32_t kBand = 8;
__device__ __forceinline__ void mx_tile(const MxProductArgs& p, uint32_t t, uint32_t& tm, uint32_t& tn) {
    const uint32_t band = t / (kBand * p.tiles_n), in = t - band * kBand * p.tiles_n;
    const uint32_t high = min(kBand, p.tiles_m - band * kBand);   // the last band may be lower
    tn = in / high;
    tm = band * kBand + in - tn * high;
}

template <int DT, int MT>
__global__ void __launch_bounds__(kMxThreads)
k_mx4_product(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
              const __grid_constant__ CUtensorMap map_sa, const __grid_constant__ CUtensorMap map_sb,
              const __grid_constant__ MxProductArgs p) {
    using T = MxTile<MT>;
    constexpr uint32_t kStages = T::kStages;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * kStages + 5];
    __shared__ uint32_t s_tmem;
    __shared__ int s_quit;
    volatile int* quit = &s_quit;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t full = smem_u32(bars), empty = full + 8 * kStages, done = empty + 8 * kStages, freed = done + 16,
                   last = freed + 16;
    if (threadIdx.x == 0) {
        s_quit = 0;
        const uint32_t held = blockIdx.x == 0 ? p.hold : 0;
        for (uint32_t i = 0; i < 2 * kStages + 2; ++i) bar_init(full + 8 * i, i < kStages && i + 1 == held ? 2 : 1);
        for (uint32_t i = 0; i < 2; ++i) bar_init(freed + 8 * i, kMxOutWarps);
        bar_init(last, 1);
        bar_init_fence();
        prefetch_map(&map_a);
        prefetch_map(&map_b);
        prefetch_map(&map_sa);
        prefetch_map(&map_sb);
    }
    if (warp == 1) tmem_alloc(smem_u32(&s_tmem), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    pdl_enter();
    const uint32_t nk = (p.k + kMxK - 1) / kMxK;

    if (warp == 0 && elect_one()) {
        Ring<kStages> r;
        uint32_t fills = 0;
        bool ok = true;
        for (uint32_t t = blockIdx.x; t < p.total && ok; t += gridDim.x) {
            uint32_t tm, tn;
            mx_tile(p, t, tm, tn);
            const int ra = static_cast<int>(tm * T::kRows), rb = static_cast<int>(tn * kMxN);
            for (uint32_t kb = 0; kb < nk; ++kb, r.next(), ++fills) {
                if (!bar_wait(empty + 8 * r.s, r.parity ^ 1, quit, kForSpace)) {   // passes at once in the first round
                    ok = false;
                    break;
                }
                const uint32_t bar = full + 8 * r.s, st = ring + r.s * T::kStage;
                const uint32_t ss = st + T::kA + T::kB;
                bar_expect(bar, T::kStage);
                copy_box(st, &map_a, static_cast<int>(kb * 128), ra, 0, bar);
                copy_box(st + T::kA, &map_b, static_cast<int>(kb * 128), rb, 0, bar);
                copy_box(ss, &map_sa, 0, static_cast<int>(8 * kb), ra >> 7, bar);
                copy_box(ss + T::kScaleA, &map_sb, 0, static_cast<int>(8 * kb), rb >> 7, bar);
            }
        }
        if (!ok) {   // the block must not leave with copies in flight
            const uint64_t t0 = now_ns();
            for (uint32_t i = fills > kStages ? fills - kStages : 0; i < fills; ++i)
                bar_drain(full + 8 * (i % kStages), (i / kStages) & 1, t0);
        }
    } else if (warp == 1 && elect_one()) {
        // e2m1 operands, power-of-two scales, 128 x 192
        constexpr uint32_t idesc =
            (1u << 7) | (1u << 10) | (static_cast<uint32_t>(kMxN >> 3) << 17) | (1u << 23) | (8u << 24);
        const uint64_t desc0 = operand_desc(ring, 0), scales0 = scale_desc(ring + T::kA + T::kB);
        Ring<kStages> r;
        uint32_t it = 0, n = 0;   // stages, and accumulators begun
        bool ok = true;
        for (uint32_t t = blockIdx.x; t < p.total && ok; t += gridDim.x, n += MT) {
            uint32_t tm, tn;
            mx_tile(p, t, tm, tn);
            const uint32_t odd = tn & 1 ? 2u : 0u;   // columns that begin with a scale tile's row 64
            for (uint32_t kb = 0; kb < nk && ok; ++kb, ++it, r.next()) {
                if (!bar_wait(full + 8 * r.s, r.parity, quit, kForData)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t da = desc0 + r.s * (T::kStage >> 4), db = da + (T::kA >> 4);
                const uint64_t ss = scales0 + r.s * (T::kStage >> 4);
                const uint32_t sf = tmem + 2 * kMxN + (it & 3) * T::kSet, sfb = sf + 8 * MT;
#pragma unroll
                for (uint32_t h = 0; h < 2; ++h) {   // per 128 values of k
#pragma unroll
                    for (uint32_t i = 0; i < MT; ++i) tc_copy_scales(sf + 8 * i + 4 * h, ss + (1024 >> 4) * i + (512 >> 4) * h);
#pragma unroll
                    for (uint32_t i = 0; i < 2; ++i)
                        tc_copy_scales(sfb + 8 * h + 4 * i, ss + (T::kScaleA >> 4) + (1024 >> 4) * i + (512 >> 4) * h);
                }
#pragma unroll
                for (uint32_t i = 0; i < MT; ++i) {
                    const uint32_t unit = n + i, acc = unit & 1, d = tmem + acc * kMxN;
                    if (kb == 0 && unit >= 2) {
                        if (!bar_wait(freed + 8 * acc, (unit / 2 - 1) & 1, quit, kForSpace)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                    }
#pragma unroll
                    for (uint32_t h = 0; h < 2; ++h) {
                        if (2 * kb + h >= p.tiles_k) break;
#pragma unroll
                        for (uint32_t j = 0; j < 2; ++j)
                            mma_mx4(d, da + (16384 >> 4) * i + (2 * h + j) * 2, db + (2 * h + j) * 2,
                                    idesc | (2 * j << 4) | (2 * j << 29), sf + 8 * i + 4 * h, sfb + 8 * h + odd,
                                    kb > 0 || h > 0 || j > 0);
                    }
                    if (kb + 1 == nk) tc_commit(done + 8 * acc);
                }
                tc_commit(empty + 8 * r.s);
            }
        }
        if (*quit) {   // tensor memory must not be freed under a product
            tc_commit(last);
            bar_drain(last, 0, now_ns());
        }
    } else if (warp >= 2) {
        const uint32_t quarter = warp & 3, part = (warp - 2) >> 2;   // 32 rows, 96 columns
        const uint32_t mine = ring + kStages * T::kStage + (warp - 2) * 2 * kMxOut;
        uint32_t n = 0, flip = 0;
        bool ok = true;
        for (uint32_t t = blockIdx.x; t < p.total && ok; t += gridDim.x) {
            uint32_t tm, tn;
            mx_tile(p, t, tm, tn);
            for (uint32_t i = 0; i < MT; ++i, ++n) {
                const uint32_t acc = n & 1;
                const uint32_t row0 = tm * T::kRows + 128 * i + quarter * 32, col0 = tn * kMxN + part * 96;
                ok = bar_wait(done + 8 * acc, (n / 2) & 1, quit);
                ok = !__any_sync(0xFFFFFFFFu, !ok);
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (uint32_t c = 0; c < 96 && row0 < p.m && col0 + c < p.n; c += 32) {   // uniform over the warp
                    const uint32_t buf = mine + flip * kMxOut;
                    flip ^= 1;
                    float v[32];
                    tmem_load32(tmem + acc * kMxN + part * 96 + c + (quarter << 21), v);
#pragma unroll
                    for (uint32_t j = 0; j < 4; ++j)
                        st_shared(buf + piece64(lane, j), narrow2<DT>(v[8 * j], v[8 * j + 1]),
                                  narrow2<DT>(v[8 * j + 2], v[8 * j + 3]), narrow2<DT>(v[8 * j + 4], v[8 * j + 5]),
                                  narrow2<DT>(v[8 * j + 6], v[8 * j + 7]));
                    __syncwarp();
                    write_rows(static_cast<unsigned short*>(p.out), p.ld, p.vec, p.m, p.n, row0, col0 + c, buf);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(freed + 8 * acc);
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    settle(quit);
    if (warp == 1) {
        tc_fence_after();
        tmem_free(tmem, 512);
    }
}

// ------------------------------------------------- product with few rows
// Up to 32 rows of A (a token, a handful): bound by reading B once, 5.7 us for
// a row against 4096 x 11008 (4.2 TB/s) and 6.6 for 32 (above 32 rows the tiles
// of 128 are faster: 8.0 us for 33 rows, 9.8 for 256).  B's rows are the tensor cores' 128 rows and A's the columns (NT of
// them), a CTA takes 128 of B's rows over a share of k, and the CTAs of a
// cluster add up their shares through shared memory, in order of rank.  The
// shares are chosen so that about two CTAs an SM have their copies in flight
// from the start.
struct MxNarrowArgs {
    uint32_t m, n;
    uint32_t tiles_k, stages;   // scale tiles along k; stages of 256 values
    uint32_t split;             // CTAs a cluster
    void* out;
    uint64_t ld;
    uint32_t hold;              // zero_debug_hold_matrix, or 0
};

constexpr int kNarrowThreads = 192, kNarrowStages = 3;
template <int NT>
struct Narrow {
    static constexpr uint32_t kB = 128 * 128, kA = NT * 128, kStage = kB + kA + 2048;   // and 1 KiB of scales each
    static constexpr size_t kSmem = 1024 + kNarrowStages * kStage;
    static constexpr uint32_t kTmem = 128;   // the accumulator and four sets of scales
    static_assert(NT + 4 * 16 <= kTmem, "tensor memory");
    static_assert(kSmem >= kLeastTmemSmem, "see tmem_alloc");
    static_assert(kNarrowStages * kStage >= NT * 512, "the partial sums take the ring's place");
};

template <int DT, int NT>
__global__ void __launch_bounds__(kNarrowThreads)
k_mx4_narrow(const __grid_constant__ CUtensorMap map_b, const __grid_constant__ CUtensorMap map_a,
             const __grid_constant__ CUtensorMap map_sb, const __grid_constant__ CUtensorMap map_sa,
             const __grid_constant__ MxNarrowArgs p) {
    using L = Narrow<NT>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * kNarrowStages + 1];
    __shared__ uint32_t s_tmem;
    __shared__ int s_quit;
    volatile int* quit = &s_quit;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = p.split > 1 ? cluster_rank() : 0, tile = blockIdx.x / p.split;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t full = smem_u32(bars), empty = full + 8 * kNarrowStages, done = empty + 8 * kNarrowStages;
    const uint32_t k0 = rank * p.stages / p.split, k1 = (rank + 1) * p.stages / p.split;
    if (threadIdx.x == 0) {
        s_quit = 0;
        const int held = blockIdx.x == 0 ? static_cast<int>(p.hold) : 0;
        for (int i = 0; i < 2 * kNarrowStages + 1; ++i) bar_init(full + 8 * i, i < kNarrowStages && i + 1 == held ? 2 : 1);
        bar_init_fence();
        prefetch_map(&map_b);
        prefetch_map(&map_a);
    }
    if (warp == 1) tmem_alloc(smem_u32(&s_tmem), L::kTmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    pdl_enter();

    if (warp == 0 && elect_one()) {
        Ring<kNarrowStages> r;
        uint32_t kb = k0;
        for (; kb < k1; ++kb, r.next()) {
            if (!bar_wait(empty + 8 * r.s, r.parity ^ 1, quit, kForSpace)) break;
            const uint32_t bar = full + 8 * r.s, st = ring + r.s * L::kStage;
            bar_expect(bar, L::kStage);
            copy_box(st, &map_b, static_cast<int>(kb * 128), static_cast<int>(tile * 128), 0, bar);
            copy_box(st + L::kB, &map_a, static_cast<int>(kb * 128), 0, 0, bar);
            copy_box(st + L::kB + L::kA, &map_sb, 0, static_cast<int>(8 * kb), static_cast<int>(tile), bar);
            copy_box(st + L::kB + L::kA + 1024, &map_sa, 0, static_cast<int>(8 * kb), 0, bar);
        }
    } else if (warp == 1 && elect_one()) {
        constexpr uint32_t idesc = (1u << 7) | (1u << 10) | (static_cast<uint32_t>(NT >> 3) << 17) | (1u << 23) | (8u << 24);
        const uint64_t desc0 = operand_desc(ring, 0), scales0 = scale_desc(ring + L::kB + L::kA);
        Ring<kNarrowStages> r;
        bool ok = true;
        for (uint32_t kb = k0; kb < k1; ++kb, r.next()) {
            if (!bar_wait(full + 8 * r.s, r.parity, quit, kForData)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint64_t db = desc0 + r.s * (L::kStage >> 4), da = db + (L::kB >> 4), ss = scales0 + r.s * (L::kStage >> 4);
            const uint32_t sf = tmem + NT + ((kb - k0) & 3) * 16;
#pragma unroll
            for (uint32_t h = 0; h < 2; ++h) {
                tc_copy_scales(sf + 4 * h, ss + (512 >> 4) * h);
                tc_copy_scales(sf + 8 + 4 * h, ss + (1024 >> 4) + (512 >> 4) * h);
            }
#pragma unroll
            for (uint32_t h = 0; h < 2; ++h) {
                if (2 * kb + h >= p.tiles_k) break;
#pragma unroll
                for (uint32_t j = 0; j < 2; ++j)
                    mma_mx4(tmem, db + (2 * h + j) * 2, da + (2 * h + j) * 2, idesc | (2 * j << 4) | (2 * j << 29),
                                sf + 4 * h, sf + 8 + 4 * h, kb > k0 || h > 0 || j > 0);
            }
            tc_commit(empty + 8 * r.s);
        }
        tc_commit(done);
        if (!ok) bar_drain(done, 0, now_ns());
    } else if (warp >= 2) {
        // partial sums [column][128 rows] where the ring was
        const bool ok = bar_wait(done, 0, quit);
        const uint32_t row = (warp & 3) * 32 + lane;
        if (!__any_sync(0xFFFFFFFFu, !ok)) {
            tc_fence_after();
#pragma unroll
            for (uint32_t c = 0; c < NT; c += 16) {
                float v[16];
                tmem_load16(tmem + c + ((warp & 3) << 21), v);
#pragma unroll
                for (uint32_t e = 0; e < 16; ++e) st_shared(ring + (c + e) * 512 + row * 4, __float_as_uint(v[e]));
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    settle(quit);
    if (warp == 1) {   // before the wait for the cluster: see tmem_alloc
        tc_fence_after();
        tmem_free(tmem, L::kTmem);
    }
    if (p.split > 1) cluster_sync();
    // this CTA's share of the rows, four at a time, for all columns
    const uint32_t rows = 128 / p.split, fours = rows / 4;   // split is a power of two, at most 8
    const uint32_t first = tile * 128 + rank * rows;
    unsigned short* out = static_cast<unsigned short*>(p.out) + first;
    const bool whole = (reinterpret_cast<uintptr_t>(out) & 7) == 0 && (p.ld & 3) == 0;
    for (uint32_t i = threadIdx.x; i < fours * p.m; i += kNarrowThreads) {
        const uint32_t c = i / fours, r = (i - c * fours) * 4;
        if (first + r >= p.n) continue;
        const uint32_t at = ring + c * 512 + (rank * rows + r) * 4;
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (uint32_t q = 0; q < p.split; ++q) {
            const float4 y = ld_cluster(cluster_addr(at, q));
            s.x += y.x; s.y += y.y; s.z += y.z; s.w += y.w;
        }
        const uint32_t lo = narrow2<DT>(s.x, s.y), hi = narrow2<DT>(s.z, s.w);
        unsigned short* to = out + c * p.ld + r;
        if (whole && first + r + 4 <= p.n) {
            *reinterpret_cast<uint2*>(to) = make_uint2(lo, hi);
        } else {
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e)
                if (first + r + e < p.n) to[e] = static_cast<unsigned short>((e < 2 ? lo : hi) >> (16 * (e & 1)));
        }
    }
    if (p.split > 1) cluster_sync();   // the others may still be reading here
}

// -------------------------------------------------------------------- host
constexpr uint64_t kMaxSide = 1ull << 30;

uint64_t mx_pitch(uint64_t cols) { return up(cols, kMxBlock) / 2; }

// Checks shared by the calls on one matrix; (rows, cols) are those of the codes.
int mx_check(int dtype, uint64_t rows, uint64_t cols, const void* codes, const void* scales) {
    if (dtype != ZERO_FP16 && dtype != ZERO_BF16) return refuse(ZERO_EINVAL, "dtype must be fp16 or bf16");
    if (rows > kMaxSide || cols > kMaxSide) return refuse(ZERO_EINVAL, "a side is longer than 2^30");
    if (rows == 0 || cols == 0) return ZERO_OK;
    if (!codes || !aligned(codes, 16)) return refuse(ZERO_EINVAL, "codes is NULL or not 16-byte aligned");
    if (!scales || !aligned(scales, 16)) return refuse(ZERO_EINVAL, "scales is NULL or not 16-byte aligned");
    return ZERO_OK;
}

// Grid of the row kernels: blocks of 8 warps down the rows, segments across.
dim3 row_grid(uint64_t rows, uint64_t cols) {
    const uint64_t per = static_cast<uint64_t>(kThreads / 32) * kMxRows, segments = up(cols, 256) / 256;
    return dim3(static_cast<unsigned>(up(rows, per) / per), static_cast<unsigned>(segments < 65535 ? segments : 65535));
}

// The map of a matrix of codes in boxes of `box_rows` rows, and of its scale
// tiles in boxes of 1 KiB (two tiles along k) by `box_tiles`.
cudaError_t mx_maps(CUtensorMap* codes_map, CUtensorMap* scales_map, const void* codes, const void* scales, uint64_t rows,
                    uint64_t k, uint32_t box_rows, uint32_t box_tiles) {
    const uint64_t pitch = mx_pitch(k), lines = up(k, 128) / 128 * 4;   // lines of 128 bytes in a row of scale tiles
    const cudaError_t e = make_map(codes_map, 1, codes, pitch, rows, 1, pitch, rows * pitch, 128, box_rows);
    return e != cudaSuccess ? e
                            : make_map(scales_map, 1, scales, 128, lines, up(rows, 128) / 128, 128, lines * 128, 128, 8,
                                       CU_TENSOR_MAP_SWIZZLE_NONE, box_tiles);
}

template <int NT>
cudaError_t narrow_of(int dtype, uint64_t m, uint64_t n, uint64_t k, const void* a_codes, const void* a_scales,
                      const void* b_codes, const void* b_scales, void* out, uint64_t ld, cudaStream_t s) {
    CUtensorMap ma, mb, sa, sb;
    int sms = 0;
    cudaError_t e;
    if ((e = sm_count(&sms)) != cudaSuccess || (e = mx_maps(&ma, &sa, a_codes, a_scales, m, k, NT, 1)) != cudaSuccess ||
        (e = mx_maps(&mb, &sb, b_codes, b_scales, n, k, 128, 1)) != cudaSuccess)
        return e;
    MxNarrowArgs p = {};
    p.m = static_cast<uint32_t>(m);
    p.n = static_cast<uint32_t>(n);
    p.tiles_k = static_cast<uint32_t>(up(k, 128) / 128);
    p.stages = static_cast<uint32_t>(up(k, kMxK) / kMxK);
    p.hold = take_matrix_hold();
    p.out = out;
    p.ld = ld;
    const uint64_t tiles = up(n, 128) / 128;
    // shares of k: up to 8, as long as all CTAs are resident at once (by their shared memory) and a share keeps two stages
    const uint64_t resident = static_cast<uint64_t>(sms) * (kSmemPerSm / (Narrow<NT>::kSmem + 1024));
    for (p.split = 1; p.split < 8 && 2 * tiles * p.split <= resident && p.stages >= 4 * p.split;) p.split *= 2;
    const dim3 grid(static_cast<unsigned>(tiles * p.split));
    if (dtype == ZERO_FP16) {
        if ((e = allow_smem<k_mx4_narrow<kFp16, NT>>(Narrow<NT>::kSmem)) != cudaSuccess) return e;
        return launch_pdl(k_mx4_narrow<kFp16, NT>, grid, kNarrowThreads, Narrow<NT>::kSmem, p.split, s, mb, ma, sb, sa, p);
    }
    if ((e = allow_smem<k_mx4_narrow<kBf16, NT>>(Narrow<NT>::kSmem)) != cudaSuccess) return e;
    return launch_pdl(k_mx4_narrow<kBf16, NT>, grid, kNarrowThreads, Narrow<NT>::kSmem, p.split, s, mb, ma, sb, sa, p);
}

}  // namespace

static std::atomic<uint32_t> g_matrix_hold{0};
uint32_t take_matrix_hold() { return g_matrix_hold.exchange(0); }

cudaError_t mx4_gave_up(cudaStream_t s, int32_t* out) { return read_gave_up(s, out); }
cudaError_t ortho_gave_up(cudaStream_t s, int32_t* out);   // zero_ortho.cu

}  // namespace zg

using namespace zg;

extern "C" {

uint64_t zero_mx4_codes_bytes(uint64_t rows, uint64_t cols) {
    return rows > kMaxSide || cols > kMaxSide ? 0 : rows * mx_pitch(cols);
}

uint64_t zero_mx4_scales_bytes(uint64_t rows, uint64_t cols) {
    return rows > kMaxSide || cols > kMaxSide ? 0 : up(rows, 128) / 128 * (up(cols, 128) / 128) * 512;
}

int zero_mx4_quantize(int dtype, uint64_t rows, uint64_t cols, const void* src16, uint64_t ld, int transpose,
                      void* codes, void* scales, void* stream) {
    nvtxRangePushA("zero_mx4_quantize");
    struct Pop { ~Pop() { nvtxRangePop(); } } pop;
    if (const int rc = mx_check(dtype, rows, cols, codes, scales)) return rc;
    if (rows == 0 || cols == 0) return ZERO_OK;
    if (!src16 || !aligned(src16, 2)) return refuse(ZERO_EINVAL, "src16 is NULL or not 2-byte aligned");
    if (ld < cols || ld > (1ull << 40)) return refuse(ZERO_EINVAL, "ld must be at least cols (and at most 2^40)");
    MxArgs a = {};
    a.src = src16;
    a.codes = static_cast<uint8_t*>(codes);
    a.scales = static_cast<uint8_t*>(scales);
    a.rows = rows;
    a.cols = cols;
    a.ld = ld;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (transpose) {
        a.pitch = mx_pitch(rows);
        a.tiles_k = up(rows, 128) / 128;
        if (a.tiles_k > 65535) return refuse(ZERO_EINVAL, "a transposed matrix has at most 65535 * 128 rows");
        const dim3 grid(static_cast<unsigned>(up(cols, 128) / 128), static_cast<unsigned>(a.tiles_k));
        e = dtype == ZERO_FP16 ? launch_pdl(k_mx4_columns<kFp16>, grid, kThreads, 0, 1, s, a)
                               : launch_pdl(k_mx4_columns<kBf16>, grid, kThreads, 0, 1, s, a);
    } else {
        a.pitch = mx_pitch(cols);
        a.tiles_k = up(cols, 128) / 128;
        const dim3 grid = row_grid(up(rows, 128), cols);
        const bool fp16 = dtype == ZERO_FP16;
        e = launch_pdl(aligned(src16, 16) && ld % 8 == 0 ? (fp16 ? k_mx4_rows<kFp16, true> : k_mx4_rows<kBf16, true>)
                                                         : (fp16 ? k_mx4_rows<kFp16, false> : k_mx4_rows<kBf16, false>),
                       grid, kThreads, 0, 1, s, a);
    }
    return e == cudaSuccess ? ZERO_OK : cuda_refuse(e, "zero_mx4_quantize");
}

int zero_mx4_dequantize(int dtype, uint64_t rows, uint64_t cols, const void* codes, const void* scales, void* out16,
                        uint64_t ld, void* stream) {
    nvtxRangePushA("zero_mx4_dequantize");
    struct Pop { ~Pop() { nvtxRangePop(); } } pop;
    if (const int rc = mx_check(dtype, rows, cols, codes, scales)) return rc;
    if (rows == 0 || cols == 0) return ZERO_OK;
    if (!out16 || !aligned(out16, 2)) return refuse(ZERO_EINVAL, "out16 is NULL or not 2-byte aligned");
    if (ld < cols || ld > (1ull << 40)) return refuse(ZERO_EINVAL, "ld must be at least cols (and at most 2^40)");
    MxArgs a = {};
    a.dst = out16;
    a.codes = static_cast<uint8_t*>(const_cast<void*>(codes));
    a.scales = static_cast<uint8_t*>(const_cast<void*>(scales));
    a.rows = rows;
    a.cols = cols;
    a.ld = ld;
    a.pitch = mx_pitch(cols);
    a.tiles_k = up(cols, 128) / 128;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool fp16 = dtype == ZERO_FP16, whole = aligned(out16, 16) && ld % 8 == 0;
    const dim3 grid = row_grid(rows, cols + (whole ? 0 : 7));
    const cudaError_t e =
        launch_pdl(whole ? (fp16 ? k_mx4_values<kFp16, true> : k_mx4_values<kBf16, true>)
                                                     : (fp16 ? k_mx4_values<kFp16, false> : k_mx4_values<kBf16, false>),
                   grid, kThreads, 0, 1, s, a);
    return e == cudaSuccess ? ZERO_OK : cuda_refuse(e, "zero_mx4_dequantize");
}

int zero_mx4_matmul(int dtype, uint64_t m, uint64_t n, uint64_t k, const void* a_codes, const void* a_scales,
                    const void* b_codes, const void* b_scales, void* out16, uint64_t ld, void* stream) {
    nvtxRangePushA("zero_mx4_matmul");
    struct Pop { ~Pop() { nvtxRangePop(); } } pop;
    if (const int rc = mx_check(dtype, m, k, a_codes, a_scales)) return rc;
    if (const int rc = mx_check(dtype, n, k, b_codes, b_scales)) return rc;
    if (m == 0 || n == 0) return ZERO_OK;
    if (!out16 || !aligned(out16, 2)) return refuse(ZERO_EINVAL, "out16 is NULL or not 2-byte aligned");
    if (ld < n || ld > (1ull << 40)) return refuse(ZERO_EINVAL, "ld must be at least n (and at most 2^40)");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (k == 0) {   // an empty sum
        e = cudaMemset2DAsync(out16, ld * 2, 0, n * 2, m, s);
        return e == cudaSuccess ? ZERO_OK : cuda_refuse(e, "zero_mx4_matmul");
    }
    if (m <= 32) {
        e = m <= 16 ? narrow_of<16>(dtype, m, n, k, a_codes, a_scales, b_codes, b_scales, out16, ld, s)
                    : narrow_of<32>(dtype, m, n, k, a_codes, a_scales, b_codes, b_scales, out16, ld, s);
        return e == cudaSuccess ? ZERO_OK : cuda_refuse(e, "zero_mx4_matmul");
    }
    int sms = 0;
    if ((e = sm_count(&sms)) != cudaSuccess) return cuda_refuse(e, "zero_mx4_matmul");
    // 256 rows a tile are cheaper a row (1224 cycles a stage against 863 for 128) unless they leave SMs idle
    const uint64_t across = up(n, kMxN) / kMxN;
    auto rounds = [&](uint64_t rows) { return (up(m, rows) / rows * across + sms - 1) / sms; };
    const bool tall = rounds(256) * 1224 <= rounds(128) * 863;
    const uint64_t rows = tall ? 256 : 128, tiles = up(m, rows) / rows * across;
    if (tiles > 0x7FFFFFFFull) return refuse(ZERO_EINVAL, "m and n are too large together");
    MxProductArgs p = {};
    p.m = static_cast<uint32_t>(m);
    p.n = static_cast<uint32_t>(n);
    p.k = static_cast<uint32_t>(k);
    p.tiles_m = static_cast<uint32_t>(up(m, rows) / rows);
    p.tiles_n = static_cast<uint32_t>(across);
    p.total = static_cast<uint32_t>(tiles);
    p.tiles_k = static_cast<uint32_t>(up(k, 128) / 128);
    p.out = out16;
    p.ld = ld;
    p.vec = aligned(out16, 16) && ld % 8 == 0;
    p.hold = take_matrix_hold();
    CUtensorMap ma, mb, sa, sb;
    if ((e = mx_maps(&ma, &sa, a_codes, a_scales, m, k, static_cast<uint32_t>(rows), tall ? 2 : 1)) != cudaSuccess ||
        (e = mx_maps(&mb, &sb, b_codes, b_scales, n, k, kMxN, 2)) != cudaSuccess)
        return cuda_refuse(e, "tensor map");
    const dim3 grid(static_cast<unsigned>(tiles < static_cast<uint64_t>(sms) ? tiles : sms));
    const bool fp16 = dtype == ZERO_FP16;
    if (tall) {
        constexpr size_t smem = MxTile<2>::kSmem;
        if ((e = allow_smem<k_mx4_product<kFp16, 2>>(smem)) == cudaSuccess &&
            (e = allow_smem<k_mx4_product<kBf16, 2>>(smem)) == cudaSuccess)
            e = launch_pdl(fp16 ? k_mx4_product<kFp16, 2> : k_mx4_product<kBf16, 2>, grid, kMxThreads, smem, 1, s, ma, mb, sa, sb, p);
    } else {
        constexpr size_t smem = MxTile<1>::kSmem;
        if ((e = allow_smem<k_mx4_product<kFp16, 1>>(smem)) == cudaSuccess &&
            (e = allow_smem<k_mx4_product<kBf16, 1>>(smem)) == cudaSuccess)
            e = launch_pdl(fp16 ? k_mx4_product<kFp16, 1> : k_mx4_product<kBf16, 1>, grid, kMxThreads, smem, 1, s, ma, mb, sa, sb, p);
    }
    return e == cudaSuccess ? ZERO_OK : cuda_refuse(e, "zero_mx4_matmul");
}

int zero_debug_hold_matrix(int64_t stage) {
    g_matrix_hold = stage < 0 || stage >= 0x7FFFFFFF ? 0u : static_cast<uint32_t>(stage) + 1u;
    return ZERO_OK;
}

int zero_matrix_status(void* stream) {
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    int32_t a = 0, b = 0;
    cudaError_t e = ortho_gave_up(s, &a);
    if (e == cudaSuccess) e = mx4_gave_up(s, &b);
    if (e != cudaSuccess) return cuda_refuse(e, "zero_matrix_status");
    if (a | b) {
        const char* what[] = {"", "space", "data", "products", "inputs"};
        const int32_t w = a ? a : b;
        return refuse(ZERO_ETIMEOUT, std::string("a bounded wait inside a kernel of ") +
                                         (a ? "zero_orthogonalize" : "zero_mx4_matmul") + " gave up, for " +
                                         what[w >= 1 && w <= 4 ? w : 0] + ": its output is incomplete");
    }
    return ZERO_OK;
}

}  // extern "C"
