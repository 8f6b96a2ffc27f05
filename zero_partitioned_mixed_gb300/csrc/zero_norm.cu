// The residual stream of a training step: dropout, and the root-mean-square
// norm with the addition (and the dropout) before it, in 16 bits or in the
// microscaled formats that the block-scaled products read; and its backward
// pass.
//
//   h  = round16(residual + dropout(x))
//   y  = h r w,  r = 1 / sqrt(mean(h^2) + eps)
//   dh = r (g - h c) + dh_in,  g = dy w,  c = r^2 mean(g h)
//   dx = dropout(dh),  dw = sum over rows of dy h r
//
// All of it is bound by HBM.  A row's statistics need the whole row before
// its first output, so a row stays in registers (packed, 16 bits a value)
// between the two: every byte is read and written once.  The norm is that of
// the stored stream, so that the backward pass, which forms r again from h
// (one more sum beside the one that it needs anyway), takes the derivative of
// what the forward pass computed.
//
// Sums are fp32: 8 to 32 values a thread, then a tree over the warp, then the
// warps in order; results repeat bit for bit (which values a thread has depends
// on the sizes, and on whether rows start on 16 bytes).

#include <cmath>
#include <cstdint>
#include <string>

#include <nvtx3/nvToolsExt.h>

#include "zero_gb300.h"
#include "zero_host.h"
#include "zero_mx.cuh"
#include "zero_tc.cuh"
#include "zero_philox.cuh"

namespace zg {
namespace {

// The weights of 256 columns: every row reads them again, from the caches.
template <int DT, bool ALIGNED>
__device__ __forceinline__ void read_weight(const unsigned short* at, int left, float (&f)[8]) {
    if constexpr (ALIGNED) {
        Loaded<true> r{make_uint4(0u, 0u, 0u, 0u)};
        if (static_cast<int>(column_of<true>(0)) < left) r.x = reinterpret_cast<const uint4*>(at)[threadIdx.x & 31];
        widen_eight<DT>(r, f);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t c = column_of<false>(e);
            f[e] = static_cast<int>(c) < left ? widen<DT>(at[c]) : 0.0f;
        }
    }
}

// ----------------------------------------------------------------- dropout
struct DropoutArgs {
    const unsigned short* src;
    unsigned short* dst;
    uint64_t cols, ld_src, ld_dst;
    uint64_t across;           // groups of 8 columns in a row
    uint64_t segments, items;  // of kDropVecs * 256 columns in a row, and in all
    DropArgs drop;
};
constexpr int kDropVecs = 4;

// Rows without gaps, of whole eights: a group's number is its place.  A thread
// takes kDropVecs groups, their loads in flight together.  HBM and the
// generator's products about even: 8192 x 4096 bf16 in 21 us (6.4 TB/s).
template <int DT>
__global__ void __launch_bounds__(kThreads) k_dropout(const __grid_constant__ DropoutArgs a) {
    pdl_enter();
    const uint64_t stream = drop_stream(a.drop), first = static_cast<uint64_t>(blockIdx.x) * kDropVecs * kThreads + threadIdx.x;
    const uint4* src = reinterpret_cast<const uint4*>(a.src);
    Loaded<true> f[kDropVecs];
#pragma unroll
    for (int i = 0; i < kDropVecs; ++i) {
        const uint64_t g = first + static_cast<uint64_t>(i) * kThreads;
        f[i].x = make_uint4(0u, 0u, 0u, 0u);
        if (g < a.across) f[i].x = __ldcs(src + g);
    }
#pragma unroll
    for (int i = 0; i < kDropVecs; ++i) {
        const uint64_t g = first + static_cast<uint64_t>(i) * kThreads;
        float x[8];
        widen_eight<DT>(f[i], x);
        if (a.drop.below) drop_eight<true>(a.drop, g, stream, x);
        uint32_t q[4];
        narrow8<DT>(x, q);
        if (g < a.across) __stcs(reinterpret_cast<uint4*>(a.dst) + g, make_uint4(q[0], q[1], q[2], q[3]));
    }
}

// Any rows: a warp takes up to kDropVecs times 256 columns of a row.
template <int DT, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) k_dropout_rows(const __grid_constant__ DropoutArgs a) {
    pdl_enter();
    const uint64_t stream = drop_stream(a.drop);
    const uint64_t item = static_cast<uint64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (item >= a.items) return;
    const uint64_t row = item / a.segments, c0 = (item - row * a.segments) * (kDropVecs * 256);
    const unsigned short* src = a.src + row * a.ld_src + c0;
    unsigned short* dst = a.dst + row * a.ld_dst + c0;
    const uint64_t group = row * a.across + c0 / 8 + (threadIdx.x & 31);
    Loaded<ALIGNED> f[kDropVecs];
#pragma unroll
    for (int i = 0; i < kDropVecs; ++i) load_eight(src + 256 * i, columns_left(a.cols, c0 + 256 * i), f[i]);
#pragma unroll
    for (int i = 0; i < kDropVecs; ++i) {
        const int left = columns_left(a.cols, c0 + 256 * i);
        if (left == 0) break;   // the same in all lanes
        float x[8];
        widen_eight<DT>(f[i], x);
        if (a.drop.below) drop_eight<ALIGNED>(a.drop, group + 32 * i, stream, x);
        uint32_t q[4];
        narrow8<DT>(x, q);
        store_eight<ALIGNED>(dst + 256 * i, left, q);
    }
}

// -------------------------------------------------------------------- norm
struct NormArgs {
    const unsigned short *x, *residual, *weight;
    unsigned short *h, *out;
    uint8_t *codes, *scales;
    uint64_t rows, cols, ld_x, ld_residual, ld_h, ld_out;
    uint64_t pitch, tiles_k;   // of the codes; 0 tiles without them
    uint64_t across;           // groups of 8 columns in a row
    float eps;
    uint32_t row_threads;      // of a row; a block has several rows where these are few
    DropArgs drop;
};

// The threads of a row: whole warps, and a block has 256 threads or one row.
struct RowThreads {
    uint32_t threads, slot, t;   // of a row; which row of the block; which of the row's threads
    __device__ __forceinline__ explicit RowThreads(uint32_t n) : threads(n), slot(threadIdx.x / n), t(threadIdx.x - slot * n) {}
    // All threads of the row have come here; each row of a block has a barrier of its own.
    __device__ __forceinline__ void sync() const {
        if (threads == 32) __syncwarp();
        else if (threads == blockDim.x) __syncthreads();
        else asm volatile("barrier.sync %0, %1;" ::"r"(slot + 1), "r"(threads) : "memory");
    }
};
// N sums over the threads of a row, in all of them.
template <int N>
__device__ __forceinline__ void row_sums(float (&s)[N], const RowThreads& row, float (*shared)[32]) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) s[k] += __shfl_xor_sync(0xFFFFFFFFu, s[k], d);
    if (row.threads == 32) return;
    const uint32_t first = (row.slot * row.threads) >> 5, warps = row.threads >> 5;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int k = 0; k < N; ++k) shared[k][threadIdx.x >> 5] = s[k];
    }
    row.sync();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        s[k] = 0.0f;
        for (uint32_t i = 0; i < warps; ++i) s[k] += shared[k][first + i];
    }
}
// A power of two to take a row's values by where its squares leave fp32
// although the row does not leave bf16 (values past 2^57 to 2^64, or the
// smallest ones with next to no eps), as their factor r shows; else 1.  For
// fp16 rows that cannot be.  (0.2 us of 61 for 8192 x 4096.)
template <int DT>
__device__ __forceinline__ float range_scale(float r) {
    return DT != kBf16 ? 1.0f : r > 0x1p30f ? 0x1p80f : r == 0.0f ? 0x1p-72f : 1.0f;
}
__device__ __forceinline__ float rsqrt_of(float sum, uint64_t cols, float eps) {
    return __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(sum, static_cast<float>(cols)), eps)));
}

// The larger magnitude; NaN where there is one.
__device__ __forceinline__ float larger(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
    return r;
}
// A warp's 256 columns of a row from c0 on, y, `left` of them inside it, to
// codes and scale words.
template <int BITS, bool ALIGNED>
__device__ __forceinline__ void write_codes(const NormArgs& a, uint64_t row, uint32_t c0, int left, float (&y)[8]) {
    if (left < 256) {   // 0 / 0 in a row of zeros, or NaN times 0, stays inside the row
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = static_cast<int>(column_of<ALIGNED>(e)) < left ? y[e] : 0.0f;
    }
    const uint32_t lane = threadIdx.x & 31;
    uint8_t* codes = a.codes + row * a.pitch;
    if constexpr (ALIGNED) {
        const uint32_t v = c0 / 8 + lane;
        // (bits of magnitudes are ordered like these, infinity and NaN above every number)
        uint32_t top = __float_as_uint(larger(larger(larger(y[0], y[1]), larger(y[2], y[3])),
                                              larger(larger(y[4], y[5]), larger(y[6], y[7]))));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));   // four lanes share a block
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        const uint32_t byte = scale_byte<BITS>(__uint_as_float(top));
        mul8(y, scale_inverse(byte));
        typename MxElement<BITS>::Eight q;
        codes8(y, q);
        if (byte == 255u) no_codes(q);
        if (v * BITS < a.pitch) *reinterpret_cast<decltype(q)*>(codes + v * BITS) = q;
        // the four blocks of a scale tile's row in one word
        uint32_t word = byte | __shfl_down_sync(0xFFFFFFFFu, byte, 4) << 8;
        word |= __shfl_down_sync(0xFFFFFFFFu, word, 8) << 16;
        if ((v & 15) == 0 && (v >> 4) < a.tiles_k)
            *reinterpret_cast<uint32_t*>(a.scales + scale_at(row, v >> 2, a.tiles_k)) = word;
    } else {   // a block is one value of each lane
        uint32_t words[2] = {0u, 0u};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(y[e]) & 0x7FFFFFFFu);
            const uint32_t byte = scale_byte<BITS>(__uint_as_float(top));
            words[e >> 2] |= byte << (8 * (e & 3));
            y[e] = __fmul_rn(y[e], scale_inverse(byte));
            const bool none = byte == 255u;
            const uint32_t c = c0 + 32 * e + lane;
            if constexpr (BITS == 8) {
                if (c < a.pitch) codes[c] = none ? 0 : static_cast<uint8_t>(codes4_e4m3(y[e], 0.0f, 0.0f, 0.0f));
            } else {
                const float next = __shfl_down_sync(0xFFFFFFFFu, y[e], 1);
                const float two[8] = {y[e], next, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
                uint32_t q;
                codes8(two, q);
                if ((lane & 1) == 0 && c / 2 < a.pitch) codes[c / 2] = none ? 0 : static_cast<uint8_t>(q);
            }
        }
        if (lane < 2 && (c0 >> 7) + lane < a.tiles_k)
            *reinterpret_cast<uint32_t*>(a.scales + scale_at(row, (c0 >> 5) + 4 * lane, a.tiles_k)) = lane == 0 ? words[0] : words[1];
    }
}

// V times 256 columns a warp, one after the other.  BITS: of the codes, or 0.
// 8192 x 4096 bf16 with residual and dropout into 16 and 8 bits: 50 us for 303
// MB (6.1 TB/s, issue slots 70 % taken); into 16 and 4 bits 50, into 16 alone
// 41, into 8 or 4 alone 46; 87 and (16 alone) 59 where one of the matrices or
// the weight does not start on 16 bytes, for then every value is an access of
// its own.
template <int BITS, int DT, int V, bool ALIGNED>
__global__ void __launch_bounds__(V == 4 ? 512 : 1024, V == 4 ? 2 : 1) k_rms_norm(const __grid_constant__ NormArgs a) {
    pdl_enter();
    __shared__ float s_sum[2][1][32];
    const RowThreads team(a.row_threads);
    const uint64_t row = static_cast<uint64_t>(blockIdx.x) * (blockDim.x / team.threads) + team.slot;
    if (row >= a.rows) {   // uniform over a row's threads; the unused rows of the last scale tiles
        if (BITS != 0 && row < (a.rows + 127) / 128 * 128)
            for (uint64_t k = team.t; k < a.tiles_k; k += team.threads)
                *reinterpret_cast<uint32_t*>(a.scales + scale_at(row, 4 * k, a.tiles_k)) = 0u;
        return;
    }
    const uint32_t c0 = (team.t >> 5) * (256 * V);   // the warp's first column
    const int cols = static_cast<int>(a.cols) - static_cast<int>(c0);
    auto left = [&](int j) { return cols - 256 * j; };   // of the row from the j-th 256 columns on
    Loaded<ALIGNED> x[V], res[V];
    uint32_t h[V][4];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        load_eight(a.x + row * a.ld_x + c0 + 256 * j, left(j), x[j]);
        if (a.residual) load_eight(a.residual + row * a.ld_residual + c0 + 256 * j, left(j), res[j]);
    }
    const uint64_t stream = drop_stream(a.drop), group = row * a.across + c0 / 8 + (threadIdx.x & 31);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        float y[8];
        widen_eight<DT>(x[j], y);
        if (a.drop.below) drop_eight<ALIGNED>(a.drop, group + 32 * j, stream, y);
        if (a.residual) {
            float s[8];
            widen_eight<DT>(res[j], s);
            add8(y, s);
        }
        narrow8<DT>(y, h[j]);   // (the values as they were where nothing was added or dropped)
    }
    float sums[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if (a.h) store_eight<ALIGNED>(a.h + row * a.ld_h + c0 + 256 * j, left(j), h[j]);
        float y[8];
        widen8<DT>(h[j], y);
        dot8(y, y, sums);
    }
    float sum[1] = {sums[0] + sums[1]};
    row_sums<1>(sum, team, s_sum[0]);
    float r = rsqrt_of(sum[0], a.cols, a.eps);
    const float scale = range_scale<DT>(r);
    if (scale != 1.0f) {   // the same in all threads of the row
        sums[0] = sums[1] = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float y[8];
            widen8<DT>(h[j], y);
            mul8(y, scale);
            dot8(y, y, sums);
        }
        sum[0] = sums[0] + sums[1];
        row_sums<1>(sum, team, s_sum[1]);
        r = __fmul_rn(rsqrt_of(sum[0], a.cols, __fmul_rn(__fmul_rn(a.eps, scale), scale)), scale);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        float y[8], f[8];
        widen8<DT>(h[j], y);
        read_weight<DT, ALIGNED>(a.weight + c0 + 256 * j, left(j), f);
        mul8(y, r);
        mul8(y, f);
        if (a.out) {
            uint32_t q[4];
            narrow8<DT>(y, q);
            store_eight<ALIGNED>(a.out + row * a.ld_out + c0 + 256 * j, left(j), q);
        }
        if constexpr (BITS != 0) write_codes<BITS, ALIGNED>(a, row, c0 + 256 * j, left(j), y);
    }
}

// ---------------------------------------------------------- norm, backward
struct NormGradArgs {
    const unsigned short *dy, *h, *weight, *dh_in;
    unsigned short *dh, *dx;
    float* partial;            // [blocks][8 * across], or NULL
    uint64_t rows, cols, ld_dy, ld_h, ld_in, ld_dh, ld_dx;
    uint64_t across;
    float eps;
    uint32_t row_threads;
    DropArgs drop;
};

// 16 bytes into shared memory.
__device__ __forceinline__ void copy16(uint4* to, const uint4* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                 ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(to))), "l"(from)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {   // all but the last N groups
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
constexpr int kGradStages = 2;
constexpr size_t grad_ring(size_t v, size_t row_threads, size_t rows) {   // bytes; a slot more a row, see below
    return 3 * kGradStages * rows * (v * row_threads + 1) * sizeof(uint4);
}
constexpr size_t kMostGradSmem = grad_ring(4, 512, 1);
static_assert(kMostGradSmem >= grad_ring(2, 64, 4) && kMostGradSmem >= grad_ring(4, 32, 8), "shared memory");

// How many values behind a 16-byte boundary a row starts.
__device__ __forceinline__ uint32_t behind(const unsigned short* row) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) >> 1) & 7u;
}

// A block takes its rows blockIdx.x, + gridDim.x, ..., and keeps its share of
// dw in registers over all of them.  The next row is on its way to shared
// memory while this one is worked on: 63 us for 8192 x 4096 bf16 with dropout
// (5.3 TB/s) against 70 with the next row in registers and 94 without.  Rows
// that start between two 16-byte boundaries are copied as the aligned pieces
// that cover them, and read from there as column_of says, two bytes at a time:
// 110 us for the same size where only the weight lies at an odd address.
template <int DT, int V, bool ALIGNED>
__global__ void __maxnreg__(V == 4 || ALIGNED ? 128 : 96) k_rms_norm_backward(const __grid_constant__ NormGradArgs a) {
    pdl_enter();
    __shared__ float s_sum[2][2][32], s_again[2][32];
    // [row of the block][stage][h, dy, dh_in][width]; at the end, with several rows: [row][8 * across] floats
    extern __shared__ __align__(16) uint4 s_rows[];
    const RowThreads team(a.row_threads);
    const uint32_t slots = blockDim.x / team.threads, lane = threadIdx.x & 31;
    const uint64_t step = static_cast<uint64_t>(gridDim.x) * slots;
    const uint64_t stream = drop_stream(a.drop);
    const uint32_t c0 = (team.t >> 5) * (256 * V), v0 = c0 / 8 + lane;   // the warp's first column, the lane's first piece
    const int cols = static_cast<int>(a.cols) - static_cast<int>(c0);
    auto left = [&](int j) { return cols - 256 * j; };   // of the row from the j-th 256 columns on
    float dw[V][8];
    Loaded<ALIGNED> w[V];
    // a row's slots: one for each eight columns, and one for the piece behind the last
    const uint32_t width = V * team.threads + 1, room = 3 * kGradStages * width;
    uint4* const mine = s_rows + team.slot * room;
    auto place = [&](uint32_t stage, int which, uint32_t v) -> uint4& { return mine[(stage * 3 + which) * width + v]; };
#pragma unroll
    for (int j = 0; j < V; ++j) {
        load_eight(a.weight + c0 + 256 * j, left(j), w[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[j][e] = 0.0f;
        if (ALIGNED && v0 + 32 * j >= a.across) {   // never copied to
#pragma unroll
            for (int i = 0; i < 3 * kGradStages; ++i) place(i / 3, i % 3, v0 + 32 * j) = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    uint64_t row = static_cast<uint64_t>(blockIdx.x) * slots + team.slot;
    auto copy_row = [&](const unsigned short* base, uint64_t ld, uint64_t row, uint32_t stage, int which) {
        if constexpr (ALIGNED) {
            const uint4* at = reinterpret_cast<const uint4*>(base + row * ld);
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (v0 + 32 * j < a.across) copy16(&place(stage, which, v0 + 32 * j), at + v0 + 32 * j);
        } else {
            const unsigned short* at = base + row * ld;
            const uint32_t m = behind(at), pieces = (m + static_cast<uint32_t>(a.cols) + 7) / 8;
            const uint4* from = reinterpret_cast<const uint4*>(at - m);
            // what is outside the matrix is not touched: the first row's first piece and the last row's last one may begin
            // or end there
            const uint4* low = reinterpret_cast<const uint4*>(base);
            const unsigned short* high = base + (a.rows - 1) * ld + a.cols;
            for (uint32_t v = team.t; v < pieces; v += team.threads) {
                if (from + v >= low && reinterpret_cast<const unsigned short*>(from + v + 1) <= high) {
                    copy16(&place(stage, which, v), from + v);
                } else {
                    unsigned short* to = reinterpret_cast<unsigned short*>(&place(stage, which, v));
#pragma unroll
                    for (uint32_t e = 0; e < 8; ++e)
                        if (8 * v + e >= m && 8 * v + e < m + a.cols) to[e] = at[8 * v + e - m];
                }
            }
        }
    };
    auto start = [&](uint64_t row, uint32_t stage) {
        if (row < a.rows) {
            copy_row(a.h, a.ld_h, row, stage, 0);
            copy_row(a.dy, a.ld_dy, row, stage, 1);
            if (a.dh_in) copy_row(a.dh_in, a.ld_in, row, stage, 2);
        }
        copy_commit();
    };
    start(row, 0);
    for (uint32_t flip = 0; row < a.rows; row += step, flip ^= 1) {   // uniform over a row's threads; flip: the stage too
        if (ALIGNED) {   // a thread reads what it copied
            start(row + step, flip ^ 1);
            copy_wait<1>();
        } else {
            copy_wait<0>();
            team.sync();   // the others' copies are there, and what they read of the row before is read
            start(row + step, flip ^ 1);
        }
        // where the row's columns begin in its slots
        const uint32_t m[3] = {ALIGNED ? 0u : behind(a.h + row * a.ld_h), ALIGNED ? 0u : behind(a.dy + row * a.ld_dy),
                               ALIGNED ? 0u : behind(a.dh_in + row * a.ld_in)};
        auto values = [&](int which, int j, float (&x)[8]) {
            if constexpr (ALIGNED) {
                widen_eight<DT>(Loaded<true>{place(flip, which, v0 + 32 * j)}, x);
            } else {
                const unsigned short* from =
                    reinterpret_cast<const unsigned short*>(&place(flip, which, 0)) + m[which] + c0 + 256 * j + lane;
                if (left(j) >= 256) {   // the same in all lanes
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = widen<DT>(from[32 * e]);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        x[e] = static_cast<int>(column_of<false>(e)) < left(j) ? widen<DT>(from[32 * e]) : 0.0f;
                }
            }
        };
        float ss[2] = {0.0f, 0.0f}, sg[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float x[8], y[8], f[8];
            values(0, j, x);
            values(1, j, y);
            widen_eight<DT>(w[j], f);
            mul8(y, f);
            dot8(x, x, ss);
            dot8(y, x, sg);
        }
        float sums[2] = {ss[0] + ss[1], sg[0] + sg[1]};
        row_sums<2>(sums, team, s_sum[flip]);
        float r = rsqrt_of(sums[0], a.cols, a.eps);
        float k = __fmul_rn(__fmul_rn(r, r), __fdiv_rn(sums[1], static_cast<float>(a.cols)));
        const float scale = range_scale<DT>(r);
        if (scale != 1.0f) {   // the same in all threads of the row
            ss[0] = ss[1] = sg[0] = sg[1] = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float x[8], y[8], f[8];
                values(0, j, x);
                values(1, j, y);
                widen_eight<DT>(w[j], f);
                mul8(x, scale);
                mul8(y, f);
                dot8(x, x, ss);
                dot8(y, x, sg);
            }
            sums[0] = ss[0] + ss[1];
            sums[1] = sg[0] + sg[1];
            row_sums<2>(sums, team, s_again);
            r = rsqrt_of(sums[0], a.cols, __fmul_rn(__fmul_rn(a.eps, scale), scale));
            k = __fmul_rn(__fmul_rn(__fmul_rn(__fdiv_rn(sums[1], static_cast<float>(a.cols)), r), r), scale);
            r = __fmul_rn(r, scale);
        }
        const uint64_t group = row * a.across + v0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            uint32_t q[4];
            float x[8], y[8], f[8];
            values(0, j, x);
            values(1, j, y);
            widen_eight<DT>(w[j], f);
            mul8(f, y);          // g
            float u[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = -k;
            fma8(x, u, f);       // g - h k
            mul8(f, r);
            mul8(x, r);
            fma8(y, x, dw[j]);
            if (a.dh_in) {
                values(2, j, x);
                add8(f, x);
            }
            narrow8<DT>(f, q);
            store_eight<ALIGNED>(a.dh + row * a.ld_dh + c0 + 256 * j, left(j), q);
            if (a.dx) {
                if (a.drop.below) drop_eight<ALIGNED>(a.drop, group + 32 * j, stream, f);
                narrow8<DT>(f, q);
                store_eight<ALIGNED>(a.dx + row * a.ld_dx + c0 + 256 * j, left(j), q);
            }
        }
    }
    copy_wait<0>();
    if (!a.partial) return;
    float* out = a.partial + static_cast<uint64_t>(blockIdx.x) * 8 * a.across;
    const uint32_t values = static_cast<uint32_t>(8 * a.across);
    float* const s_dw = reinterpret_cast<float*>(s_rows);
    if (slots > 1) __syncthreads();   // the rows are done with; their shares of dw take their place
    float* to = slots > 1 ? s_dw + team.slot * values : out;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if constexpr (ALIGNED) {
            if (v0 + 32 * j >= a.across) continue;
            float4* at = reinterpret_cast<float4*>(to + 8 * (v0 + 32 * j));
            at[0] = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
            at[1] = make_float4(dw[j][4], dw[j][5], dw[j][6], dw[j][7]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t c = c0 + 256 * j + column_of<false>(e);
                if (c < values) to[c] = dw[j][e];
            }
        }
    }
    if (slots == 1) return;
    __syncthreads();
    for (uint32_t c = threadIdx.x; c < values; c += blockDim.x) {
        float s = 0.0f;
        for (uint32_t i = 0; i < slots; ++i) s += s_dw[i * values + c];
        out[c] = s;
    }
}

// dw from the blocks' shares: a warp takes 32 columns of every 32nd share, the
// 32 warps' sums are added in order.
template <int DT>
__global__ void __launch_bounds__(1024) k_norm_dweight(const float* partial, uint64_t parts, uint64_t width, uint64_t cols,
                                                       unsigned short* dw) {
    pdl_enter();
    __shared__ float s[32][33];
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint64_t c = static_cast<uint64_t>(blockIdx.x) * 32 + lane;
    float sum = 0.0f;
    if (c < cols) {
#pragma unroll 10
        for (uint64_t p = warp; p < parts; p += 32) sum += partial[p * width + c];
    }
    s[warp][lane] = sum;
    __syncthreads();
    if (warp != 0 || c >= cols) return;
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += s[i][lane];
    dw[c] = static_cast<unsigned short>(narrow<DT>(sum));
}

// -------------------------------------------------------------------- host
constexpr uint64_t kMaxRows = 1ull << 30, kMaxLd = 1ull << 40;
constexpr uint64_t kMostOddRow = 1ull << 34;   // columns of dropout's rows that are not whole eights from 16 bytes on, without gaps

struct Matrix {
    const char* name;
    const void* at;
    uint64_t ld;
    bool needed;
};
// Refusals of the matrices of a call; whether all rows start on 16 bytes and are whole eights.
int check_matrices(const Matrix* m, int count, uint64_t cols, bool& whole) {
    whole = cols % 8 == 0;
    for (int i = 0; i < count; ++i) {
        if (!m[i].at) {
            if (m[i].needed) return refuse(ZERO_EINVAL, std::string(m[i].name) + " is NULL");
            continue;
        }
        if (!aligned(m[i].at, 2)) return refuse(ZERO_EINVAL, std::string(m[i].name) + " is not 2-byte aligned");
        if (m[i].ld < cols || m[i].ld > kMaxLd)
            return refuse(ZERO_EINVAL, "ld of " + std::string(m[i].name) + " must be at least cols (and at most 2^40)");
        whole = whole && aligned(m[i].at, 16) && m[i].ld % 8 == 0;
    }
    return ZERO_OK;
}
int check_sizes(int dtype, uint64_t rows, uint64_t cols, uint64_t most) {
    if (dtype != ZERO_FP16 && dtype != ZERO_BF16) return refuse(ZERO_EINVAL, "dtype must be fp16 or bf16");
    if (rows > kMaxRows) return refuse(ZERO_EINVAL, "more than 2^30 rows");
    if (cols > most) return refuse(ZERO_EINVAL, "more than " + std::to_string(most) + " columns");
    return ZERO_OK;
}

template <int BITS, int DT, int V>
cudaError_t launch_norm(const NormArgs& a, bool whole, unsigned blocks, unsigned threads, cudaStream_t s) {
    constexpr bool kOdd = V == 4;   // at odd strides a thread has no more than 2 (norm_shape)
    static_assert(2 * 8 * 1024 >= ZERO_MAX_NORM_COLS, "rows at odd strides in 2 eights a thread");
    return launch_pdl(whole ? k_rms_norm<BITS, DT, V, true> : k_rms_norm<BITS, DT, V, kOdd>, dim3(blocks), threads, 0, 1, s, a);
}
template <int BITS, int DT>
cudaError_t launch_norm(const NormArgs& a, int v, bool whole, unsigned blocks, unsigned threads, cudaStream_t s) {
    return v == 1   ? launch_norm<BITS, DT, 1>(a, whole, blocks, threads, s)
           : v == 2 ? launch_norm<BITS, DT, 2>(a, whole, blocks, threads, s)
                    : launch_norm<BITS, DT, 4>(a, whole, blocks, threads, s);
}
template <int DT, int V>
cudaError_t launch_norm_grad(const NormGradArgs& a, bool whole, unsigned blocks, unsigned threads, size_t smem, cudaStream_t s) {
    const size_t ring = grad_ring(V, a.row_threads, threads / a.row_threads);
    if (ring > smem) smem = ring;
    cudaError_t e;
    if ((e = allow_smem<k_rms_norm_backward<DT, V, true>>(kMostGradSmem)) != cudaSuccess ||
        (e = allow_smem<k_rms_norm_backward<DT, V, false>>(kMostGradSmem)) != cudaSuccess)
        return e;
    return launch_pdl(whole ? k_rms_norm_backward<DT, V, true> : k_rms_norm_backward<DT, V, false>, dim3(blocks), threads, smem,
                      1, s, a);
}
template <int DT>
cudaError_t launch_norm_grad(const NormGradArgs& a, int v, bool whole, unsigned blocks, unsigned threads, size_t smem,
                             cudaStream_t s) {
    return v == 1   ? launch_norm_grad<DT, 1>(a, whole, blocks, threads, smem, s)
           : v == 2 ? launch_norm_grad<DT, 2>(a, whole, blocks, threads, smem, s)
                    : launch_norm_grad<DT, 4>(a, whole, blocks, threads, smem, s);
}

// How a row of `groups` eights lies over threads: `v` eights each, as near to
// `most_v` (a power of two) as leaves no more than three tenths of the threads'
// places empty, and more where the threads would be over `most`.  (Fewer eights
// a thread cost more than some empty places: 8192 x 768 forward 17 us at 4 of
// which a quarter is empty, 22 at 1 of which none is; backward 18 and 27.)
struct RowShape {
    int v;
    unsigned row_threads, rows;   // rows: of a block at a time
};
RowShape row_shape(uint64_t groups, int most_v, unsigned most) {
    auto of = [&](int v) {
        const unsigned n = static_cast<unsigned>(up((groups + v - 1) / v, 32));
        return RowShape{v, n, n < kThreads ? kThreads / n : 1u};
    };
    RowShape r = of(most_v);
    for (int v = most_v; v >= 1; v /= 2) {
        const RowShape s = of(v);
        if (s.row_threads > most) break;
        const auto places = [](const RowShape& x) { return static_cast<uint64_t>(x.v) * x.row_threads; };
        if (places(s) < places(r) || r.row_threads > most) r = s;
        if (10 * groups >= 7 * places(r)) break;
    }
    while (r.row_threads > most) r = of(2 * r.v);
    return r;
}
// Few rows finish sooner with more threads each; many are cheaper a row with
// fewer: 64 x 4096 with dropout into 8 bits 4.2, 4.4 and 5.3 us at 1, 2 and 4
// eights a thread, 608 x 4096 9.6, 8.2 and 9.5, 8192 x 4096 76, 68 and 61 (all
// with the codes read back again).  Rows at odd strides hold a register a value
// and stop at 2: 4001 x 5003 84 us, 87 at 1 and 92 at 4, when that was chosen,
// and 76 now.  Without the reading back, at 1, 2 and 4: 400 x 768 2.6, 3.1 and
// 3.9, 608 x 2048 3.7, 4.1 and 5.2, 1300 x 768 4.5, 4.9 and 4.7, 1300 x 2048
// 7.6, 6.4 and 8.1, 8192 x 768 17.7, 15.0 and 13.3, 8192 x 2048 39.6, 29.7 and
// 26.7: beside a limit the rule is up to a quarter off.
RowShape norm_shape(uint64_t rows, uint64_t groups, bool whole) {
    const int v = !whole ? (rows >= 1216 ? 2 : 1) : rows >= 1216 ? 4 : rows >= 304 ? 2 : 1;
    return row_shape(groups, v, v == 4 ? 512 : 1024);
}
// Backward: blocks enough that an SM has some 512 threads (a block of 160, of
// which two an SM left it idle, took 96 us for 6057 x 2187), and few enough
// that their shares of dw are little beside the rows.  At 1, 2 and 4 eights a
// thread: 8192 x 768 20.9, 20.4 and 17.3 us, 8192 x 1024 25.6, 21.1 and 18.8,
// 8001 x 1003 50, 35 and 30, 8192 x 2048 44, 36.3 and 36.8, 8192 x 4096 97,
// 63.6 and 65.6, 6057 x 2187 66, 54 and 83.  Between them the rule is not the
// best everywhere: 8192 x 1536 takes 39 with 2 and 31 with 4, 8192 x 3000 71
// and 60, 8192 x 8192 138 and 114.
constexpr unsigned kGradBlocks = 304;   // two an SM
RowShape grad_shape(uint64_t rows, uint64_t cols) {
    return row_shape((cols + 7) / 8, rows < kGradBlocks ? 1 : cols <= 1024 ? 4 : 2, 512);
}
uint64_t grad_blocks(uint64_t rows, const RowShape& r) {
    const unsigned threads = r.rows * r.row_threads;
    const uint64_t b = (rows + r.rows - 1) / r.rows, most = kGradBlocks / 2 * (threads <= 160 ? 4 : threads <= 192 ? 3 : 2);
    return b < most ? b : most;
}

}  // namespace
}  // namespace zg

using namespace zg;

extern "C" {

int zero_dropout(int dtype, uint64_t rows, uint64_t cols, const void* src16, uint64_t ld_src, void* out16, uint64_t ld_out,
                 const zero_dropout_t* dropout, void* stream) {
    nvtxRangePushA("zero_dropout");
    struct Pop { ~Pop() { nvtxRangePop(); } } pop;
    DropoutArgs a = {};
    bool whole = true;
    if (const int rc = check_sizes(dtype, rows, cols, 1ull << 40)) return rc;
    if (const int rc = drop_args(a.drop, dropout)) return rc;
    if (rows == 0 || cols == 0) return ZERO_OK;
    const Matrix m[] = {{"src16", src16, ld_src, true}, {"out16", out16, ld_out, true}};
    if (const int rc = check_matrices(m, 2, cols, whole)) return rc;
    // one long row has the same groups; past kMostOddRow only where rows may be that long
    if (cols % 8 == 0 && ld_src == cols && ld_out == cols && rows <= (whole ? 1ull << 40 : kMostOddRow) / cols) {
        cols *= rows;
        rows = 1;
        ld_src = ld_out = cols;
    }
    a.src = static_cast<const unsigned short*>(src16);
    a.dst = static_cast<unsigned short*>(out16);
    a.cols = cols;
    a.ld_src = ld_src;
    a.ld_dst = ld_out;
    a.across = (cols + 7) / 8;
    a.segments = (cols + kDropVecs * 256 - 1) / (kDropVecs * 256);
    if (a.across > (1ull << 40) / rows) return refuse(ZERO_EINVAL, "rows and cols are too large together");
    a.items = rows * a.segments;
    const bool one = whole && rows == 1, fp16 = dtype == ZERO_FP16;
    if (!one && cols > kMostOddRow) return refuse(ZERO_EINVAL, "rows of more than 2^34 values must be aligned and without gaps");
    const uint64_t per = one ? kDropVecs * kThreads : kThreads / 32;
    const uint64_t blocks = ((one ? a.across : a.items) + per - 1) / per;
    if (blocks > 0x7FFFFFFFull) return refuse(ZERO_EINVAL, "rows and cols are too large together");
    const cudaError_t e = launch_pdl(one     ? (fp16 ? k_dropout<kFp16> : k_dropout<kBf16>)
                                     : whole ? (fp16 ? k_dropout_rows<kFp16, true> : k_dropout_rows<kBf16, true>)
                                             : (fp16 ? k_dropout_rows<kFp16, false> : k_dropout_rows<kBf16, false>),
                                     dim3(static_cast<unsigned>(blocks)), kThreads, 0, 1, static_cast<cudaStream_t>(stream), a);
    return e == cudaSuccess ? ZERO_OK : cuda_refuse(e, "zero_dropout");
}

int zero_rms_norm(int dtype, uint64_t rows, uint64_t cols, const void* x16, uint64_t ld_x, const void* residual16,
                  uint64_t ld_residual, const void* weight16, float eps, const zero_dropout_t* dropout, void* h16, uint64_t ld_h,
                  void* out16, uint64_t ld_out, int bits, void* codes, void* scales, void* stream) {
    nvtxRangePushA("zero_rms_norm");
    struct Pop { ~Pop() { nvtxRangePop(); } } pop;
    NormArgs a = {};
    bool whole = true;
    if (const int rc = check_sizes(dtype, rows, cols, ZERO_MAX_NORM_COLS)) return rc;
    if (const int rc = drop_args(a.drop, dropout)) return rc;
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return refuse(ZERO_EINVAL, "eps must be finite and >= 0");
    if (bits != 0 && bits != 4 && bits != 8) return refuse(ZERO_EINVAL, "bits must be 0, 4 or 8");
    if (rows == 0 || cols == 0) return ZERO_OK;
    const Matrix m[] = {{"x16", x16, ld_x, true}, {"weight16", weight16, up(cols, 8), true}, {"residual16", residual16, ld_residual, false},
                        {"h16", h16, ld_h, false}, {"out16", out16, ld_out, false}};
    if (const int rc = check_matrices(m, 5, cols, whole)) return rc;
    if (bits) {
        if (!codes || !aligned(codes, 16)) return refuse(ZERO_EINVAL, "codes is NULL or not 16-byte aligned");
        if (!scales || !aligned(scales, 16)) return refuse(ZERO_EINVAL, "scales is NULL or not 16-byte aligned");
    } else if (!h16 && !out16) {
        return refuse(ZERO_EINVAL, "there is nothing to write: h16, out16 and bits are 0");
    }
    a.x = static_cast<const unsigned short*>(x16);
    a.residual = static_cast<const unsigned short*>(residual16);
    a.weight = static_cast<const unsigned short*>(weight16);
    a.h = static_cast<unsigned short*>(h16);
    a.out = static_cast<unsigned short*>(out16);
    a.codes = static_cast<uint8_t*>(codes);
    a.scales = static_cast<uint8_t*>(scales);
    a.rows = rows;
    a.cols = cols;
    a.ld_x = ld_x;
    a.ld_residual = ld_residual;
    a.ld_h = ld_h;
    a.ld_out = ld_out;
    a.across = (cols + 7) / 8;
    a.pitch = up(cols, kMxBlock) * bits / 8;
    a.tiles_k = bits ? up(cols, 128) / 128 : 0;
    a.eps = eps;
    const RowShape r = norm_shape(rows, bits ? 16 * a.tiles_k : a.across, whole);
    a.row_threads = r.row_threads;
    const uint64_t all = bits ? up(rows, 128) : rows;
    const unsigned blocks = static_cast<unsigned>((all + r.rows - 1) / r.rows);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool fp16 = dtype == ZERO_FP16;
    const auto of = bits == 0   ? (fp16 ? launch_norm<0, kFp16> : launch_norm<0, kBf16>)
                    : bits == 4 ? (fp16 ? launch_norm<4, kFp16> : launch_norm<4, kBf16>)
                                : (fp16 ? launch_norm<8, kFp16> : launch_norm<8, kBf16>);
    const cudaError_t e = of(a, r.v, whole, blocks, r.rows * r.row_threads, s);
    return e == cudaSuccess ? ZERO_OK : cuda_refuse(e, "zero_rms_norm");
}

uint64_t zero_rms_norm_backward_workspace_bytes(uint64_t rows, uint64_t cols) {
    if (rows == 0 || cols == 0 || rows > kMaxRows || cols > ZERO_MAX_NORM_COLS) return 0;
    return grad_blocks(rows, grad_shape(rows, cols)) * up(cols, 8) * sizeof(float);
}

int zero_rms_norm_backward(int dtype, uint64_t rows, uint64_t cols, const void* dy16, uint64_t ld_dy, const void* h16,
                           uint64_t ld_h, const void* weight16, float eps, const void* dh_in16, uint64_t ld_in, void* dh16,
                           uint64_t ld_dh, const zero_dropout_t* dropout, void* dx16, uint64_t ld_dx, void* dweight16,
                           void* workspace, uint64_t workspace_bytes, void* stream) {
    nvtxRangePushA("zero_rms_norm_backward");
    struct Pop { ~Pop() { nvtxRangePop(); } } pop;
    NormGradArgs a = {};
    bool whole = true;
    if (const int rc = check_sizes(dtype, rows, cols, ZERO_MAX_NORM_COLS)) return rc;
    if (const int rc = drop_args(a.drop, dropout)) return rc;
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return refuse(ZERO_EINVAL, "eps must be finite and >= 0");
    if (cols == 0) return ZERO_OK;
    if (dweight16 && !aligned(dweight16, 2)) return refuse(ZERO_EINVAL, "dweight16 is not 2-byte aligned");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (rows == 0) {   // an empty sum
        e = dweight16 ? cudaMemsetAsync(dweight16, 0, cols * 2, s) : cudaSuccess;
        return e == cudaSuccess ? ZERO_OK : cuda_refuse(e, "zero_rms_norm_backward");
    }
    const Matrix m[] = {{"dy16", dy16, ld_dy, true}, {"h16", h16, ld_h, true}, {"weight16", weight16, up(cols, 8), true},
                        {"dh_in16", dh_in16, ld_in, false}, {"dh16", dh16, ld_dh, true}, {"dx16", dx16, ld_dx, false}};
    if (const int rc = check_matrices(m, 6, cols, whole)) return rc;
    if (dx16 && dx16 == dh16) return refuse(ZERO_EINVAL, "dx16 and dh16 must be two matrices");
    if (dweight16) {
        if (!workspace || !aligned(workspace, 16)) return refuse(ZERO_EINVAL, "workspace is NULL or not 16-byte aligned");
        if (workspace_bytes < zero_rms_norm_backward_workspace_bytes(rows, cols))
            return refuse(ZERO_EINVAL, "workspace is smaller than zero_rms_norm_backward_workspace_bytes()");
    }
    const RowShape r = grad_shape(rows, cols);
    const unsigned blocks = static_cast<unsigned>(grad_blocks(rows, r));
    a.dy = static_cast<const unsigned short*>(dy16);
    a.h = static_cast<const unsigned short*>(h16);
    a.weight = static_cast<const unsigned short*>(weight16);
    a.dh_in = static_cast<const unsigned short*>(dh_in16);
    a.dh = static_cast<unsigned short*>(dh16);
    a.dx = static_cast<unsigned short*>(dx16);
    a.partial = dweight16 ? static_cast<float*>(workspace) : nullptr;
    a.rows = rows;
    a.cols = cols;
    a.ld_dy = ld_dy;
    a.ld_h = ld_h;
    a.ld_in = ld_in;
    a.ld_dh = ld_dh;
    a.ld_dx = ld_dx;
    a.across = (cols + 7) / 8;
    a.eps = eps;
    a.row_threads = r.row_threads;
    const size_t smem = r.rows > 1 && dweight16 ? r.rows * 8 * a.across * sizeof(float) : 0;   // less than the rows' own
    const bool fp16 = dtype == ZERO_FP16;
    e = fp16 ? launch_norm_grad<kFp16>(a, r.v, whole, blocks, r.rows * r.row_threads, smem, s)
             : launch_norm_grad<kBf16>(a, r.v, whole, blocks, r.rows * r.row_threads, smem, s);
    if (e == cudaSuccess && dweight16)
        e = launch_pdl(fp16 ? k_norm_dweight<kFp16> : k_norm_dweight<kBf16>, dim3(static_cast<unsigned>((cols + 31) / 32)), 1024, 0,
                       1, s, static_cast<const float*>(a.partial), static_cast<uint64_t>(blocks), 8 * a.across, cols,
                       static_cast<unsigned short*>(dweight16));
    return e == cudaSuccess ? ZERO_OK : cuda_refuse(e, "zero_rms_norm_backward");
}

}  // extern "C"
