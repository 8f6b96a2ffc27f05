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
// Sums are fp32: 8 to 64 values a thread, then a tree over the warp, then the
// warps in order; results repeat bit for bit.

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

// 8 weights: every row reads them again, from the caches.
template <bool ALIGNED>
__device__ __forceinline__ void read_weight(const RowIn<ALIGNED>& r, uint32_t v, int valid, uint32_t (&w)[4]) {
    if constexpr (ALIGNED) {
        const uint4 x = valid > 0 ? r.first[v] : make_uint4(0u, 0u, 0u, 0u);
        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    } else {
        read8<false>(r, v, valid, w);
    }
}
// How many of a thread's 8 columns from group v on lie inside the row.
template <bool ALIGNED>
__device__ __forceinline__ int inside(uint32_t v, uint32_t cols) {
    const int left = static_cast<int>(cols) - static_cast<int>(8 * v);
    return ALIGNED ? (left > 0 ? 8 : 0) : left > 8 ? 8 : left;
}

// f(0), f(1), ... f(N - 1), the number known to the compiler.
template <int N, typename F, int... I>
__device__ __forceinline__ void each(F&& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F&& f) {
    each<N>(f, std::make_integer_sequence<int, N>{});
}

// ----------------------------------------------------------------- dropout
struct DropoutArgs {
    const unsigned short* src;
    unsigned short* dst;
    uint64_t rows, cols, ld_src, ld_dst;
    uint64_t across;           // groups of 8 columns in a row
    uint64_t segments, items;  // of kDropVecs * 256 columns in a row, and in all
    DropArgs drop;
};
constexpr int kDropVecs = 4;

template <int DT>
__device__ __forceinline__ void drop_one(const DropoutArgs& a, uint64_t group, uint64_t stream, const uint32_t (&w)[4],
                                         uint32_t (&q)[4]) {
    float x[8];
    widen8<DT>(w, x);
    if (a.drop.below) drop8(a.drop, group, stream, x);
    narrow8<DT>(x, q);
}

// Rows without gaps, of whole eights: a group's number is its place.  A thread
// takes kDropVecs groups, their loads in flight together.  HBM and the
// generator's products about even: 8192 x 4096 bf16 in 21 us (6.4 TB/s).
template <int DT>
__global__ void __launch_bounds__(kThreads) k_dropout(const __grid_constant__ DropoutArgs a) {
    pdl_enter();
    const uint64_t stream = drop_stream(a.drop), first = static_cast<uint64_t>(blockIdx.x) * kDropVecs * kThreads + threadIdx.x;
    const uint4* src = reinterpret_cast<const uint4*>(a.src);
    Fetched<true> f[kDropVecs];
#pragma unroll
    for (int i = 0; i < kDropVecs; ++i) {
        const uint64_t g = first + static_cast<uint64_t>(i) * kThreads;
        fetch8(RowIn<true>{src + g}, 0, g < a.across ? 8 : 0, f[i]);
    }
#pragma unroll
    for (int i = 0; i < kDropVecs; ++i) {
        const uint64_t g = first + static_cast<uint64_t>(i) * kThreads;
        const uint32_t w[4] = {f[i].x.x, f[i].x.y, f[i].x.z, f[i].x.w};
        uint32_t q[4];
        drop_one<DT>(a, g, stream, w, q);
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
    const uint64_t row = item / a.segments;
    const uint32_t v0 = static_cast<uint32_t>(item - row * a.segments) * (kDropVecs * 32) + (threadIdx.x & 31);
    const RowIn<ALIGNED> in = row_in<ALIGNED>(a.src, row, a.ld_src, a.rows, a.cols);
    RowOut<ALIGNED> out(a.dst + row * a.ld_dst);
    Fetched<ALIGNED> f[kDropVecs];
    auto valid = [&](uint32_t v) { return values_left(a.cols, 8ull * v); };
#pragma unroll
    for (int i = 0; i < kDropVecs; ++i) fetch8(in, v0 + 32 * i, valid(v0 + 32 * i), f[i]);
    each<kDropVecs>([&](auto step) {
        constexpr int i = decltype(step)::value;
        const uint32_t v = v0 + 32 * i;
        if (8ull * (v & ~31u) >= a.cols) return;   // the same in all lanes
        uint32_t w[4], q[4];
        finish8(in, v, valid(v), f[i], w);
        drop_one<DT>(a, row * a.across + v, stream, w, q);
        out.template put<i == 0, i + 1 == kDropVecs>(v, valid(v), valid(v + 1), q);
    });
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
__device__ __forceinline__ float rsqrt_of(float sum, uint64_t cols, float eps) {
    return __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(sum, static_cast<float>(cols)), eps)));
}

// The larger magnitude; NaN where there is one.
__device__ __forceinline__ float larger(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
    return r;
}
// One warp's 256 values of a row: 8 a lane, y, to codes and scale words.
// v: the lane's group of 8 columns, `valid` of them inside the row.
template <int BITS>
__device__ __forceinline__ void write_codes(const NormArgs& a, uint64_t row, uint32_t v, int valid, float (&y)[8]) {
    if (valid < 8) {   // 0 / 0 in a row of zeros, or NaN times 0, stays inside the row
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = e < valid ? y[e] : 0.0f;
    }
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
    if (v * BITS < a.pitch) *reinterpret_cast<decltype(q)*>(a.codes + row * a.pitch + v * BITS) = q;
    // the four blocks of a scale tile's row in one word
    uint32_t word = byte | __shfl_down_sync(0xFFFFFFFFu, byte, 4) << 8;
    word |= __shfl_down_sync(0xFFFFFFFFu, word, 8) << 16;
    if ((v & 15) == 0 && (v >> 4) < a.tiles_k)
        *reinterpret_cast<uint32_t*>(a.scales + scale_at(row, v >> 2, a.tiles_k)) = word;
}

// V groups of 8 columns a thread, those of a row in steps of its threads.
// BITS: of the codes, or 0.  ALIGNED: every row of every matrix starts on 16
// bytes and is whole eights.
template <int BITS, int DT, int V, bool ALIGNED>
__global__ void __launch_bounds__(V == 4 ? 512 : 1024, V == 4 && ALIGNED ? 2 : 1) k_rms_norm(const __grid_constant__ NormArgs a) {
    pdl_enter();
    __shared__ float s_sum[1][32];
    const RowThreads team(a.row_threads);
    const uint32_t threads = team.threads, t = team.t;
    const uint64_t row = static_cast<uint64_t>(blockIdx.x) * (blockDim.x / threads) + team.slot;
    if (row >= a.rows) {   // uniform over a row's threads; the unused rows of the last scale tiles
        if (BITS != 0 && row < (a.rows + 127) / 128 * 128)
            for (uint64_t k = t; k < a.tiles_k; k += threads)
                *reinterpret_cast<uint32_t*>(a.scales + scale_at(row, 4 * k, a.tiles_k)) = 0u;
        return;
    }
    const uint32_t cols = static_cast<uint32_t>(a.cols), v0 = (t >> 5) * (32 * V) + (t & 31);
    Fetched<ALIGNED> x[V], res[V];
    uint32_t h[V][4];
    const RowIn<ALIGNED> in_x = row_in<ALIGNED>(a.x, row, a.ld_x, a.rows, a.cols);
    const RowIn<ALIGNED> in_res = row_in<ALIGNED>(a.residual, row, a.ld_residual, a.rows, a.cols);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint32_t v = v0 + 32 * j;
        fetch8(in_x, v, inside<ALIGNED>(v, cols), x[j]);
        if (a.residual) fetch8(in_res, v, inside<ALIGNED>(v, cols), res[j]);
    }
    const uint64_t stream = drop_stream(a.drop), group = row * a.across;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint32_t v = v0 + 32 * j;
        finish8(in_x, v, inside<ALIGNED>(v, cols), x[j], h[j]);
        if (a.residual || a.drop.below) {
            float y[8];
            widen8<DT>(h[j], y);
            if (a.drop.below) drop8(a.drop, group + v, stream, y);
            if (a.residual) {
                uint32_t q[4];
                finish8(in_res, v, inside<ALIGNED>(v, cols), res[j], q);
                float s[8];
                widen8<DT>(q, s);
                add8(y, s);
            }
            narrow8<DT>(y, h[j]);
        }
    }
    float sums[2] = {0.0f, 0.0f};
    RowOut<ALIGNED> out_h(a.h + row * a.ld_h), out_y(a.out + row * a.ld_out);
    each<V>([&](auto step) {
        constexpr int j = decltype(step)::value;
        const uint32_t v = v0 + 32 * j;
        if (a.h) out_h.template put<j == 0, j + 1 == V>(v, inside<ALIGNED>(v, cols), inside<ALIGNED>(v + 1, cols), h[j]);
        float y[8];
        widen8<DT>(h[j], y);
        dot8(y, y, sums);
    });
    float sum[1] = {sums[0] + sums[1]};
    row_sums<1>(sum, team, s_sum);
    const float r = rsqrt_of(sum[0], a.cols, a.eps);
    const RowIn<ALIGNED> in_w = row_in<ALIGNED>(a.weight, 0, 0, 1, a.cols);
    each<V>([&](auto step) {
        constexpr int j = decltype(step)::value;
        const uint32_t v = v0 + 32 * j;
        const int valid = inside<ALIGNED>(v, cols);
        uint32_t w[4];
        read_weight<ALIGNED>(in_w, v, valid, w);
        float y[8], f[8];
        widen8<DT>(h[j], y);
        widen8<DT>(w, f);
        mul8(y, r);
        mul8(y, f);
        if (a.out) {
            uint32_t q[4];
            narrow8<DT>(y, q);
            out_y.template put<j == 0, j + 1 == V>(v, valid, inside<ALIGNED>(v + 1, cols), q);
        }
        if constexpr (BITS != 0) write_codes<BITS>(a, row, v, valid, y);
    });
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

// A block takes its rows blockIdx.x, + gridDim.x, ..., and keeps its share of dw in registers over all of them.  The next
// row is on its way to shared memory while this one is worked on: 62 us for
// 8192 x 4096 bf16 with dropout (5.4 TB/s) against 70 with the next row in
// registers and 94 without.  Rows that start between two 16-byte boundaries
// are copied as the aligned pieces that cover them; a thread then needs two
// neighbouring pieces, of which another thread copied the second.
template <int DT, int V, bool ALIGNED>
__global__ void __maxnreg__(V == 4 || ALIGNED ? 128 : 96) k_rms_norm_backward(const __grid_constant__ NormGradArgs a) {
    pdl_enter();
    __shared__ float s_sum[2][2][32];
    // [row of the block][stage][h, dy, dh_in][width]; at the end, with several rows: [row][8 * across] floats
    extern __shared__ __align__(16) uint4 s_rows[];
    const RowThreads team(a.row_threads);
    const uint32_t threads = team.threads, t = team.t, slot = team.slot, slots = blockDim.x / threads;
    const uint64_t step = static_cast<uint64_t>(gridDim.x) * slots;
    const uint64_t stream = drop_stream(a.drop);
    const uint32_t cols = static_cast<uint32_t>(a.cols), v0 = (t >> 5) * (32 * V) + (t & 31);
    float dw[V][8];
    uint32_t w[V][4];
    // a row's slots: one for each group, and one for the piece behind the last
    const uint32_t width = V * threads + 1, room = 3 * kGradStages * width;
    uint4* const mine = s_rows + slot * room;
    auto place = [&](uint32_t stage, int which, uint32_t v) -> uint4& { return mine[(stage * 3 + which) * width + v]; };
    const RowIn<ALIGNED> in_w = row_in<ALIGNED>(a.weight, 0, 0, 1, a.cols);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint32_t v = v0 + 32 * j;
        const int valid = inside<ALIGNED>(v, cols);
        read_weight<ALIGNED>(in_w, v, valid, w[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[j][e] = 0.0f;
        if (ALIGNED && valid <= 0) {   // never copied to
#pragma unroll
            for (int i = 0; i < 3 * kGradStages; ++i) place(i / 3, i % 3, v) = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    uint64_t row = static_cast<uint64_t>(blockIdx.x) * slots + slot;
    auto copy_row = [&](const RowIn<ALIGNED>& r, uint32_t stage, int which) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const uint32_t v = v0 + 32 * j;
            const int valid = inside<ALIGNED>(v, cols);
            if (valid <= 0) continue;
            if constexpr (ALIGNED) {
                copy16(&place(stage, which, v), r.first + v);
            } else {
                if (r.m == 8u) {   // the first row or the last one
                    place(stage, which, v) = read_some(r.row + 8ull * v, valid);
                } else {
                    copy16(&place(stage, which, v), r.first + v);
                    if (v + 1 == a.across && valid > 8 - static_cast<int>(r.m)) copy16(&place(stage, which, v + 1), r.first + v + 1);
                }
            }
        }
    };
    auto start = [&](uint64_t row, uint32_t stage) {
        if (row < a.rows) {
            copy_row(row_in<ALIGNED>(a.h, row, a.ld_h, a.rows, a.cols), stage, 0);
            copy_row(row_in<ALIGNED>(a.dy, row, a.ld_dy, a.rows, a.cols), stage, 1);
            if (a.dh_in) copy_row(row_in<ALIGNED>(a.dh_in, row, a.ld_in, a.rows, a.cols), stage, 2);
        }
        copy_commit();
    };
    start(row, 0);
    for (uint32_t flip = 0; row < a.rows; row += step, flip ^= 1) {   // uniform over a row's threads; flip: the stage too
        if (ALIGNED) {
            start(row + step, flip ^ 1);
            copy_wait<1>();
        } else {
            copy_wait<0>();
            team.sync();   // the others' copies are there, and what they read of the row before is read
            start(row + step, flip ^ 1);
        }
        auto values = [&](int which, int j, const unsigned short* base, uint64_t ld, uint32_t (&q)[4]) {
            const uint32_t v = v0 + 32 * j;
            const uint4 p = place(flip, which, v);
            q[0] = p.x; q[1] = p.y; q[2] = p.z; q[3] = p.w;
            if constexpr (!ALIGNED) {
                const uint4 n = place(flip, which, v + 1);
                const uint32_t own[4] = {p.x, p.y, p.z, p.w}, next[4] = {n.x, n.y, n.z, n.w};
                shift_halves(own, next, row_in<false>(base, row, ld, a.rows, a.cols).m & 7u, q);
                const int valid = inside<false>(v, cols);
                if (valid < 8) clear_tail(q, valid);
            }
        };
        // what had to be put together is kept for the second pass, where there are registers for it
        constexpr bool kHold = !ALIGNED && V <= 2;
        uint32_t held[kHold ? V : 1][2][4];
        float ss[2] = {0.0f, 0.0f}, sg[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < V; ++j) {
            uint32_t p[4], q[4];
            values(0, j, a.h, a.ld_h, p);
            values(1, j, a.dy, a.ld_dy, q);
            if constexpr (kHold) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    held[j][0][i] = p[i];
                    held[j][1][i] = q[i];
                }
            }
            float x[8], y[8], f[8];
            widen8<DT>(p, x);
            widen8<DT>(q, y);
            widen8<DT>(w[j], f);
            mul8(y, f);
            dot8(x, x, ss);
            dot8(y, x, sg);
        }
        float sums[2] = {ss[0] + ss[1], sg[0] + sg[1]};
        row_sums<2>(sums, team, s_sum[flip]);
        const float r = rsqrt_of(sums[0], a.cols, a.eps);
        const float k = __fmul_rn(__fmul_rn(r, r), __fdiv_rn(sums[1], static_cast<float>(a.cols)));
        const uint64_t group = row * a.across;
        RowOut<ALIGNED> out_h(a.dh + row * a.ld_dh), out_x(a.dx + row * a.ld_dx);
        each<V>([&](auto number) {
            constexpr int j = decltype(number)::value;
            const uint32_t v = v0 + 32 * j;
            const int valid = inside<ALIGNED>(v, cols), next = inside<ALIGNED>(v + 1, cols);
            uint32_t q[4];
            float x[8], y[8], f[8];
            if constexpr (kHold) {
                widen8<DT>(held[j][0], x);
                widen8<DT>(held[j][1], y);
            } else {
                values(0, j, a.h, a.ld_h, q);
                widen8<DT>(q, x);
                values(1, j, a.dy, a.ld_dy, q);
                widen8<DT>(q, y);
            }
            widen8<DT>(w[j], f);
            mul8(f, y);          // g
            float u[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = -k;
            fma8(x, u, f);       // g - h k
            mul8(f, r);
            mul8(x, r);
            fma8(y, x, dw[j]);
            if (a.dh_in) {
                values(2, j, a.dh_in, a.ld_in, q);
                widen8<DT>(q, x);
                add8(f, x);
            }
            narrow8<DT>(f, q);
            out_h.template put<j == 0, j + 1 == V>(v, valid, next, q);
            if (a.dx) {
                if (a.drop.below) drop8(a.drop, group + v, stream, f);
                narrow8<DT>(f, q);
                out_x.template put<j == 0, j + 1 == V>(v, valid, next, q);
            }
        });
    }
    copy_wait<0>();
    if (!a.partial) return;
    float* out = a.partial + static_cast<uint64_t>(blockIdx.x) * 8 * a.across;
    if (slots == 1) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const uint32_t v = v0 + 32 * j;
            if (v >= a.across) continue;
            float4* to = reinterpret_cast<float4*>(out + 8 * v);
            to[0] = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
            to[1] = make_float4(dw[j][4], dw[j][5], dw[j][6], dw[j][7]);
        }
        return;
    }
    // the rows' shares, added in their order, where the rows were
    __syncthreads();
    float* const s_dw = reinterpret_cast<float*>(s_rows);
    const uint32_t values = static_cast<uint32_t>(8 * a.across);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint32_t v = v0 + 32 * j;
        if (v >= a.across) continue;
        float4* to = reinterpret_cast<float4*>(s_dw + slot * values + 8 * v);
        to[0] = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
        to[1] = make_float4(dw[j][4], dw[j][5], dw[j][6], dw[j][7]);
    }
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
    return launch_pdl(whole ? k_rms_norm<BITS, DT, V, true> : k_rms_norm<BITS, DT, V, false>, dim3(blocks), threads, 0, 1, s, a);
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
// eights a thread, 608 x 4096 9.6, 8.2 and 9.5, 8192 x 4096 76, 68 and 61.
RowShape norm_shape(uint64_t rows, uint64_t groups) {
    const int v = rows >= 1216 ? 4 : rows >= 304 ? 2 : 1;
    return row_shape(groups, v, v == 4 ? 512 : 1024);
}
constexpr unsigned kGradBlocks = 304;   // two an SM
RowShape grad_shape(uint64_t cols) { return row_shape((cols + 7) / 8, cols <= 1024 ? 4 : 2, 512); }
uint64_t grad_blocks(uint64_t rows, const RowShape& r) {
    const uint64_t b = (rows + r.rows - 1) / r.rows;
    return b < kGradBlocks ? b : kGradBlocks;
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
    if (cols % 8 == 0 && ld_src == cols && ld_out == cols && rows <= (1ull << 40) / cols) {   // one long row has the same groups
        cols *= rows;
        rows = 1;
        ld_src = ld_out = cols;
    }
    a.src = static_cast<const unsigned short*>(src16);
    a.dst = static_cast<unsigned short*>(out16);
    a.rows = rows;
    a.cols = cols;
    a.ld_src = ld_src;
    a.ld_dst = ld_out;
    a.across = (cols + 7) / 8;
    a.segments = (cols + kDropVecs * 256 - 1) / (kDropVecs * 256);
    if (a.across > (1ull << 40) / rows) return refuse(ZERO_EINVAL, "rows and cols are too large together");
    a.items = rows * a.segments;
    const bool one = whole && rows == 1, fp16 = dtype == ZERO_FP16;
    if (!one && cols > (1ull << 34)) return refuse(ZERO_EINVAL, "rows of more than 2^34 values must be aligned and without gaps");
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
    const RowShape r = norm_shape(rows, bits ? 16 * a.tiles_k : a.across);
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
    return grad_blocks(rows, grad_shape(cols)) * up(cols, 8) * sizeof(float);
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
    const RowShape r = grad_shape(cols);
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
