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
#include "zero_philox.cuh"

namespace zg {
namespace {

// 8 weights: every row reads them again, from the caches.
template <bool ALIGNED>
__device__ __forceinline__ void read_weight(const unsigned short* weight, uint64_t c, int valid, uint64_t cols,
                                            uint32_t (&w)[4]) {
    if (ALIGNED) {
        const uint4 x = valid > 0 ? *reinterpret_cast<const uint4*>(weight + c) : make_uint4(0u, 0u, 0u, 0u);
        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    } else {
        read8<false>(weight, c, valid, cols, w);
    }
}
// How many of a thread's 8 columns from group v on lie inside the row.
template <bool ALIGNED>
__device__ __forceinline__ int inside(uint32_t v, uint32_t cols) {
    const int left = static_cast<int>(cols) - static_cast<int>(8 * v);
    return ALIGNED ? (left > 0 ? 8 : 0) : left > 8 ? 8 : left;
}

// ----------------------------------------------------------------- dropout
struct DropoutArgs {
    const unsigned short* src;
    unsigned short* dst;
    uint64_t rows, cols, ld_src, ld_dst;
    uint64_t across, groups;   // groups of 8 columns in a row, and in all
    DropArgs drop;
};
constexpr int kDropVecs = 4;

// A thread takes kDropVecs groups, their loads in flight together.  ONE_ROW:
// a group's number is its place (rows without gaps, of whole eights).
template <int DT, bool ALIGNED, bool ONE_ROW>
__global__ void __launch_bounds__(kThreads) k_dropout(const __grid_constant__ DropoutArgs a) {
    pdl_enter();
    const uint64_t stream = drop_stream(a.drop), first = static_cast<uint64_t>(blockIdx.x) * kDropVecs * kThreads + threadIdx.x;
    uint32_t w[kDropVecs][4];
    uint64_t row[kDropVecs], c[kDropVecs];
    int valid[kDropVecs];
#pragma unroll
    for (int i = 0; i < kDropVecs; ++i) {
        const uint64_t g = first + static_cast<uint64_t>(i) * kThreads;
        // one division of 32 bits where that is enough
        row[i] = ONE_ROW ? 0ull : a.groups <= 0xFFFFFFFFull ? static_cast<uint32_t>(g) / static_cast<uint32_t>(a.across) : g / a.across;
        c[i] = 8 * (g - row[i] * a.across);
        valid[i] = g >= a.groups ? 0 : ALIGNED ? 8 : values_left(a.cols, c[i]);
        read8<ALIGNED>(a.src, row[i] * a.ld_src + c[i], valid[i], (a.rows - 1) * a.ld_src + a.cols, w[i]);
    }
#pragma unroll
    for (int i = 0; i < kDropVecs; ++i) {
        float v[8];
        widen8<DT>(w[i], v);
        if (a.drop.below) drop8(a.drop, first + static_cast<uint64_t>(i) * kThreads, stream, v);
        uint32_t q[4];
        narrow8<DT>(v, q);
        store8<ALIGNED>(a.dst + row[i] * a.ld_dst, c[i], valid[i], q);
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
    int by_warp;               // a row a warp; else a row a block
    DropArgs drop;
};

// N sums over the threads of a row, in all of them.
template <int N>
__device__ __forceinline__ void row_sums(float (&s)[N], bool by_warp, float (*shared)[32]) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) s[k] += __shfl_xor_sync(0xFFFFFFFFu, s[k], d);
    if (by_warp) return;
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int k = 0; k < N; ++k) shared[k][warp] = s[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        s[k] = 0.0f;
        for (int i = 0; i < warps; ++i) s[k] += shared[k][i];
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
__global__ void __launch_bounds__(1024) k_rms_norm(const __grid_constant__ NormArgs a) {
    pdl_enter();
    __shared__ float s_sum[1][32];
    const uint32_t threads = a.by_warp ? 32u : blockDim.x, t = a.by_warp ? threadIdx.x & 31u : threadIdx.x;
    const uint64_t row = a.by_warp ? static_cast<uint64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= a.rows) {   // uniform over a row's threads; the unused rows of the last scale tiles
        if (BITS != 0 && row < (a.rows + 127) / 128 * 128)
            for (uint64_t k = t; k < a.tiles_k; k += threads)
                *reinterpret_cast<uint32_t*>(a.scales + scale_at(row, 4 * k, a.tiles_k)) = 0u;
        return;
    }
    const uint32_t cols = static_cast<uint32_t>(a.cols);
    uint32_t h[V][4];
    const uint64_t at_x = row * a.ld_x, total_x = (a.rows - 1) * a.ld_x + a.cols;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint32_t v = j * threads + t;
        read8<ALIGNED>(a.x, at_x + 8 * v, inside<ALIGNED>(v, cols), total_x, h[j]);
    }
    if (a.residual || a.drop.below) {
        uint32_t r[V][4];
        if (a.residual) {
            const uint64_t at_r = row * a.ld_residual, total_r = (a.rows - 1) * a.ld_residual + a.cols;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const uint32_t v = j * threads + t;
                read8<ALIGNED>(a.residual, at_r + 8 * v, inside<ALIGNED>(v, cols), total_r, r[j]);
            }
        }
        const uint64_t stream = drop_stream(a.drop), group = row * a.across + t;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float y[8];
            widen8<DT>(h[j], y);
            if (a.drop.below) drop8(a.drop, group + j * threads, stream, y);
            if (a.residual) {
                float s[8];
                widen8<DT>(r[j], s);
                add8(y, s);
            }
            narrow8<DT>(y, h[j]);
        }
    }
    float sums[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint32_t v = j * threads + t;
        if (a.h) store8<ALIGNED>(a.h + row * a.ld_h, 8 * v, inside<ALIGNED>(v, cols), h[j]);
        float y[8];
        widen8<DT>(h[j], y);
        dot8(y, y, sums);
    }
    float sum[1] = {sums[0] + sums[1]};
    row_sums<1>(sum, a.by_warp, s_sum);
    const float r = rsqrt_of(sum[0], a.cols, a.eps);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint32_t v = j * threads + t;
        const int valid = inside<ALIGNED>(v, cols);
        uint32_t w[4];
        read_weight<ALIGNED>(a.weight, 8 * v, valid, a.cols, w);
        float y[8], f[8];
        widen8<DT>(h[j], y);
        widen8<DT>(w, f);
        mul8(y, r);
        mul8(y, f);
        if (a.out) {
            uint32_t q[4];
            narrow8<DT>(y, q);
            store8<ALIGNED>(a.out + row * a.ld_out, 8 * v, valid, q);
        }
        if constexpr (BITS != 0) write_codes<BITS>(a, row, v, valid, y);
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
    int by_warp;
    DropArgs drop;
};

// A block takes rows blockIdx.x, + gridDim.x, ... (by_warp: one a warp at a
// time), and keeps its share of dw in registers over all of them.  The next
// row's loads are in flight while this one's sums are formed.
template <int DT, int V, bool ALIGNED>
__global__ void __launch_bounds__(512) k_rms_norm_backward(const __grid_constant__ NormGradArgs a) {
    pdl_enter();
    __shared__ float s_sum[2][2][32];
    extern __shared__ __align__(16) float s_dw[];   // by_warp: [warps][8 * across]
    const uint32_t threads = a.by_warp ? 32u : blockDim.x, t = a.by_warp ? threadIdx.x & 31u : threadIdx.x;
    const uint32_t slots = a.by_warp ? blockDim.x >> 5 : 1u, slot = a.by_warp ? threadIdx.x >> 5 : 0u;
    const uint64_t step = static_cast<uint64_t>(gridDim.x) * slots;
    const uint64_t stream = drop_stream(a.drop);
    const uint64_t total_y = (a.rows - 1) * a.ld_dy + a.cols, total_h = (a.rows - 1) * a.ld_h + a.cols,
                   total_i = (a.rows - 1) * a.ld_in + a.cols;
    const uint32_t cols = static_cast<uint32_t>(a.cols);
    constexpr bool kAhead = V <= 2;   // registers for two rows
    float dw[V][8];
    uint32_t h[V][4], dy[V][4], in[V][4];
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[j][e] = 0.0f;
    auto load = [&](uint64_t row, uint32_t (&h)[V][4], uint32_t (&dy)[V][4], uint32_t (&in)[V][4]) {
        const uint64_t at_h = row * a.ld_h, at_y = row * a.ld_dy, at_i = row * a.ld_in;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const uint32_t v = j * threads + t;
            const int valid = inside<ALIGNED>(v, cols);
            read8<ALIGNED>(a.h, at_h + 8 * v, valid, total_h, h[j]);
            read8<ALIGNED>(a.dy, at_y + 8 * v, valid, total_y, dy[j]);
            if (a.dh_in) read8<ALIGNED>(a.dh_in, at_i + 8 * v, valid, total_i, in[j]);
        }
    };
    uint64_t row = static_cast<uint64_t>(blockIdx.x) * slots + slot;
    if (row < a.rows) load(row, h, dy, in);
    for (int flip = 0; row < a.rows; row += step, flip ^= 1) {   // uniform over a row's threads
        float ss[2] = {0.0f, 0.0f}, sg[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const uint32_t v = j * threads + t;
            uint32_t w[4];
            read_weight<ALIGNED>(a.weight, 8 * v, inside<ALIGNED>(v, cols), a.cols, w);
            float x[8], y[8], f[8];
            widen8<DT>(h[j], x);
            widen8<DT>(dy[j], y);
            widen8<DT>(w, f);
            mul8(y, f);
            dot8(x, x, ss);
            dot8(y, x, sg);
        }
        constexpr int N = kAhead ? V : 1;
        uint32_t h2[N][4], dy2[N][4], in2[N][4];
        const bool more = row + step < a.rows;
        if constexpr (kAhead) {
            if (more) load(row + step, h2, dy2, in2);
        }
        float sums[2] = {ss[0] + ss[1], sg[0] + sg[1]};
        row_sums<2>(sums, a.by_warp, s_sum[flip]);
        const float r = rsqrt_of(sums[0], a.cols, a.eps);
        const float k = __fmul_rn(__fmul_rn(r, r), __fdiv_rn(sums[1], static_cast<float>(a.cols)));
        const uint64_t group = row * a.across + t;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const uint32_t v = j * threads + t;
            const int valid = inside<ALIGNED>(v, cols);
            uint32_t w[4];
            read_weight<ALIGNED>(a.weight, 8 * v, valid, a.cols, w);
            float x[8], y[8], f[8];
            widen8<DT>(h[j], x);
            widen8<DT>(dy[j], y);
            widen8<DT>(w, f);
            mul8(f, y);          // g
            float u[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = -k;
            fma8(x, u, f);       // g - h k
            mul8(f, r);
            mul8(x, r);
            fma8(y, x, dw[j]);
            if (a.dh_in) {
                widen8<DT>(in[j], x);
                add8(f, x);
            }
            uint32_t q[4];
            narrow8<DT>(f, q);
            store8<ALIGNED>(a.dh + row * a.ld_dh, 8 * v, valid, q);
            if (a.dx) {
                if (a.drop.below) drop8(a.drop, group + j * threads, stream, f);
                narrow8<DT>(f, q);
                store8<ALIGNED>(a.dx + row * a.ld_dx, 8 * v, valid, q);
            }
        }
        if constexpr (kAhead) {
            if (more) {
#pragma unroll
                for (int j = 0; j < V; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        h[j][i] = h2[j][i];
                        dy[j][i] = dy2[j][i];
                        in[j][i] = in2[j][i];
                    }
            }
        } else if (more) {
            load(row + step, h, dy, in);
        }
    }
    if (!a.partial) return;
    float* out = a.partial + static_cast<uint64_t>(blockIdx.x) * 8 * a.across;
    if (!a.by_warp) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const uint64_t v = j * threads + t;
            if (v >= a.across) continue;
            float4* to = reinterpret_cast<float4*>(out + 8 * v);
            to[0] = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
            to[1] = make_float4(dw[j][4], dw[j][5], dw[j][6], dw[j][7]);
        }
        return;
    }
    // the warps' shares, added in their order
    const uint32_t width = static_cast<uint32_t>(8 * a.across);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint32_t v = j * threads + t;
        if (v >= a.across) continue;
        float4* to = reinterpret_cast<float4*>(s_dw + slot * width + 8 * v);
        to[0] = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
        to[1] = make_float4(dw[j][4], dw[j][5], dw[j][6], dw[j][7]);
    }
    __syncthreads();
    for (uint32_t c = threadIdx.x; c < width; c += blockDim.x) {
        float s = 0.0f;
        for (uint32_t i = 0; i < slots; ++i) s += s_dw[i * width + c];
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
#pragma unroll 4
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

// How a row of `groups` eights lies over threads: a warp up to 128 of them,
// else a block of `most` threads or fewer with `v` eights each.
struct RowShape {
    int v, by_warp;
    unsigned threads;   // of a block
    unsigned rows;      // of a block at a time
};
RowShape row_shape(uint64_t groups, unsigned least_v, unsigned most) {
    RowShape r;
    if (groups <= 128) {
        r.by_warp = 1;
        r.v = groups <= 32 ? 1 : groups <= 64 ? 2 : 4;
        r.threads = kThreads;
        r.rows = kThreads / 32;
        return r;
    }
    r.by_warp = 0;
    r.v = static_cast<int>(least_v);
    while (groups > static_cast<uint64_t>(r.v) * most) r.v *= 2;
    r.threads = static_cast<unsigned>(up((groups + r.v - 1) / r.v, 32));
    r.rows = 1;
    return r;
}
constexpr unsigned kGradBlocks = 304;   // two an SM
RowShape grad_shape(uint64_t cols) { return row_shape((cols + 7) / 8, 2, 512); }
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
    if (a.across > (1ull << 40) / rows) return refuse(ZERO_EINVAL, "rows and cols are too large together");
    a.groups = rows * a.across;
    const uint64_t blocks = (a.groups + kDropVecs * kThreads - 1) / (kDropVecs * kThreads);
    if (blocks > 0x7FFFFFFFull) return refuse(ZERO_EINVAL, "rows and cols are too large together");
    const bool fp16 = dtype == ZERO_FP16;
    const cudaError_t e = launch_pdl(whole && rows == 1 ? (fp16 ? k_dropout<kFp16, true, true> : k_dropout<kBf16, true, true>)
                                     : whole            ? (fp16 ? k_dropout<kFp16, true, false> : k_dropout<kBf16, true, false>)
                                                        : (fp16 ? k_dropout<kFp16, false, false> : k_dropout<kBf16, false, false>),
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
    const RowShape r = row_shape(bits ? 16 * a.tiles_k : a.across, 1, 1024);
    a.by_warp = r.by_warp;
    const uint64_t all = bits ? up(rows, 128) : rows;
    const unsigned blocks = static_cast<unsigned>((all + r.rows - 1) / r.rows);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool fp16 = dtype == ZERO_FP16;
    const auto of = bits == 0   ? (fp16 ? launch_norm<0, kFp16> : launch_norm<0, kBf16>)
                    : bits == 4 ? (fp16 ? launch_norm<4, kFp16> : launch_norm<4, kBf16>)
                                : (fp16 ? launch_norm<8, kFp16> : launch_norm<8, kBf16>);
    const cudaError_t e = of(a, r.v, whole, blocks, r.threads, s);
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
    a.by_warp = r.by_warp;
    const size_t smem = r.by_warp && dweight16 ? r.rows * 8 * a.across * sizeof(float) : 0;   // 32 KiB at most
    const bool fp16 = dtype == ZERO_FP16;
    e = fp16 ? launch_norm_grad<kFp16>(a, r.v, whole, blocks, r.threads, smem, s)
             : launch_norm_grad<kBf16>(a, r.v, whole, blocks, r.threads, smem, s);
    if (e == cudaSuccess && dweight16)
        e = launch_pdl(fp16 ? k_norm_dweight<kFp16> : k_norm_dweight<kBf16>, dim3(static_cast<unsigned>((cols + 31) / 32)), 1024, 0,
                       1, s, static_cast<const float*>(a.partial), static_cast<uint64_t>(blocks), 8 * a.across, cols,
                       static_cast<unsigned short*>(dweight16));
    return e == cudaSuccess ? ZERO_OK : cuda_refuse(e, "zero_rms_norm_backward");
}

}  // extern "C"
