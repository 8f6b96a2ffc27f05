// Newton-Schulz orthogonalisation of a batch of matrices (the update of the
// Muon optimiser) on the tensor cores.
//
//   X_0 = G / ||G||_F;   A = X X^T (over the shorter side);
//   X <- p(A) X,  p(A) = a I + b A + c A^2      (`steps` times)
//
// Precision.  Every stored matrix is fp16 times a fixed power of two (11 bits
// of significand against bf16's 8, at the same tensor rate); the products
// accumulate in fp32.  G itself is exact in that form up to one power of two.
// The rounding that costs most is that of X while its small singular values
// are still small, so the first two steps do not form X_1 at all: with
// B = p(A) they compose A_1 = (B A) B and Q = p(A_1) B, and X_2 = Q X_0.
// Against 64 bits the result is off by 1.0e-3 to 1.9e-3 (2-norm, gradients
// of low rank over noise, 64 x 64 to 768 x 2048), about what its rounding to
// bf16 costs (1.7e-3); rounding every X gives up to 3.2e-3 and bf16
// throughout 1e-2 to 2.5e-2.
//
// Work.  All products but the last of a step are symmetric: only tiles on or
// below the diagonal are computed and each is written twice.  For the
// shorter side s and the longer l, the first two steps cost s^2 l + 5 s^3 +
// 2 s^2 l and each further one 3 s^2 l + s^3 multiply-adds (times one; a
// plain product would be s^2 l times two).  X is never transposed: a tall
// matrix takes its Gram matrix from MN-major operands and is multiplied from
// the right, a wide one the other way around.

#include <cmath>
#include <cstdint>
#include <string>

#include <nvtx3/nvToolsExt.h>

#include "zero_gb300.h"
#include "zero_tc.cuh"

namespace zg {
namespace {

constexpr int kMaxMatrices = ZERO_MAX_MATRICES;

// Storage scales (all powers of two): entries of X and A are at most a
// little over 1, those of p(A) and Q at most a^2 or so.
constexpr float kScaleX = 8192.0f, kScaleA = 4096.0f, kScaleB = 128.0f;

// ------------------------------------------------------- norm and packing
// A matrix is read in units of one row's segment of kSegment columns, one
// warp a unit: 8 loads of 8 values a lane in flight.
constexpr int kSegment = 2048;
constexpr int kPartials = 256;   // partial sums of squares of one matrix, at most
constexpr int kPackWarps = kThreads / 32;

struct PackArgs {
    const void* src[kMaxMatrices];
    uint64_t rows, cols, ld, pitch;
    uint64_t segments, units;   // segments a row; units a matrix
    int vec;                    // every row starts on 16 bytes
    int partials;
    double* partial;            // [batch][kPartials]
    float* g0;                  // [batch]
    __half* x0;                 // [batch][rows][pitch]
};

// A lane's values of unit `u`: vals[8 k + e] is column seg + 256 k + 8 lane + e.
template <int DT>
__device__ __forceinline__ void load_unit(const PackArgs& a, int b, uint64_t u, uint64_t& row, uint64_t& col0,
                                          float (&v)[64]) {
    const int lane = threadIdx.x & 31;
    row = u / a.segments;
    col0 = (u - row * a.segments) * kSegment;
    const unsigned short* src = static_cast<const unsigned short*>(a.src[b]) + row * a.ld;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint64_t c = col0 + 256 * k + 8 * lane;
        if (a.vec && c + 8 <= a.cols) {
            const uint4 x = __ldg(reinterpret_cast<const uint4*>(src + c));
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) v[8 * k + e] = widen<DT>((w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[8 * k + e] = c + e < a.cols ? widen<DT>(__ldg(src + c + e)) : 0.0f;
        }
    }
}

// Sum of squares: 64 values in fp32, everything above in fp64.  Values whose
// squares could leave fp32's range are squared in fp64.
template <int DT>
__global__ void __launch_bounds__(kThreads) k_ortho_norm(const __grid_constant__ PackArgs a) {
    pdl_enter();
    const int b = blockIdx.y;
    double acc = 0.0;
    for (uint64_t u = static_cast<uint64_t>(blockIdx.x) * kPackWarps + (threadIdx.x >> 5); u < a.units;
         u += static_cast<uint64_t>(gridDim.x) * kPackWarps) {
        uint64_t row, col0;
        float v[64];
        load_unit<DT>(a, b, u, row, col0, v);
        float s = 0.0f, top = 0.0f;
#pragma unroll
        for (int i = 0; i < 64; ++i) {
            s = __fmaf_rn(v[i], v[i], s);
            top = fmaxf(top, fabsf(v[i]));
        }
        if (!(s < INFINITY) || !(top < 0x1p60f) || (top > 0.0f && top < 0x1p-50f)) {
            double d = 0.0;
#pragma unroll 8
            for (int i = 0; i < 64; ++i) d = fma(static_cast<double>(v[i]), static_cast<double>(v[i]), d);
            acc += d;
        } else {
            acc += static_cast<double>(s);
        }
    }
    const double t = block_sum(acc);
    if (threadIdx.x == 0) a.partial[static_cast<uint64_t>(b) * kPartials + blockIdx.x] = t;
}

// X0 = G 2^k in fp16, k such that ||G|| 2^k lies in [2^12, 2^13), and g0 =
// 1 / (||G|| 2^k), which the products that read X0 take into their scale.
// A zero matrix gives g0 = 0; infinities and NaN give a NaN g0.
template <int DT>
__global__ void __launch_bounds__(kThreads) k_ortho_pack(const __grid_constant__ PackArgs a) {
    pdl_enter();
    __shared__ float s_mul[2];
    const int b = blockIdx.y;
    const double t = block_sum(static_cast<int>(threadIdx.x) < a.partials
                                   ? a.partial[static_cast<uint64_t>(b) * kPartials + threadIdx.x]
                                   : 0.0);
    if (threadIdx.x == 0) {
        const double norm = sqrt(t);
        int e = 0;
        float g = 0.0f;
        if (norm > 0.0 && norm < INFINITY) {
            frexp(norm, &e);   // norm = f 2^e, f in [1/2, 1)
            e = 13 - e;
            g = static_cast<float>(1.0 / ldexp(norm, e));
        } else if (!(norm == 0.0)) {
            g = NAN;
        }
        // 2^e as two factors, each a normal fp32 number
        s_mul[0] = ldexpf(1.0f, e / 2);
        s_mul[1] = ldexpf(1.0f, e - e / 2);
        if (blockIdx.x == 0) a.g0[b] = g;
    }
    __syncthreads();
    const float m0 = s_mul[0], m1 = s_mul[1];
    for (uint64_t u = static_cast<uint64_t>(blockIdx.x) * kPackWarps + (threadIdx.x >> 5); u < a.units;
         u += static_cast<uint64_t>(gridDim.x) * kPackWarps) {
        uint64_t row, col0;
        float v[64];
        load_unit<DT>(a, b, u, row, col0, v);
        __half* out = a.x0 + (static_cast<uint64_t>(b) * a.rows + row) * a.pitch;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint64_t c = col0 + 256 * k + 8 * (threadIdx.x & 31);
            if (c < a.cols) {   // the row's padding up to 8 columns is written as zeros
                uint32_t q[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    q[e] = pack_half2(v[8 * k + 2 * e] * m0 * m1, v[8 * k + 2 * e + 1] * m0 * m1);
                *reinterpret_cast<uint4*>(out + c) = make_uint4(q[0], q[1], q[2], q[3]);
            }
        }
    }
}

// ---------------------------------------------------------------- products
// One product of every matrix of the batch, out = epilogue(A B^T): A has the
// output's rows, B its columns, both over `depth`.
enum Epi : int {
    kScale,   // out = f acc
    kPoly,    // out = f acc + f_lin lin + f_diag I
    kFinal,   // bf16, into the caller's matrices: out = f acc
};

struct ProductArgs {
    uint32_t rows, cols, depth;
    uint32_t tiles_n, tiles, total;   // tiles a row, a matrix, all
    __half* out;
    const __half* lin;
    uint32_t pitch;          // of out and lin
    uint64_t stride;         // between matrices of out and lin
    float f_acc, f_lin, f_diag;
    const float* g0;         // further factor g0[b]^g_power, or null
    int g_power;
    void* dst[kMaxMatrices]; // kFinal
    uint64_t dst_ld;
    int dst_vec;             // every row of dst starts on 16 bytes
};

constexpr int kBlockM = 128, kBlockK = 64;
constexpr int kProductThreads = 192;   // copies, products, 4 warps of epilogue

__host__ __device__ constexpr int stages_of(int bn) { return bn == 256 ? 4 : 6; }
__host__ __device__ constexpr uint32_t stage_bytes(int bn) { return (kBlockM + bn) * kBlockK * 2u; }
__host__ __device__ constexpr size_t product_smem(int bn) { return 1024 + static_cast<size_t>(stages_of(bn)) * stage_bytes(bn); }

// Warp 0 copies operand tiles into a ring of stages, warp 1 issues the
// products, warps 2 to 5 read finished accumulators; two accumulators in
// tensor memory, so that the epilogue of one tile runs under the products of
// the next.
template <int BN, bool A_MN, bool B_MN, int EPI, bool SYM>
__global__ void __launch_bounds__(kProductThreads)
k_ortho_product(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                const __grid_constant__ ProductArgs p) {
    constexpr int kStages = stages_of(BN);
    constexpr uint32_t kStageBytes = stage_bytes(BN), kABytes = kBlockM * kBlockK * 2;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * kStages + 4];
    __shared__ uint32_t s_tmem;
    __shared__ int s_quit;
    volatile int* quit = &s_quit;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t full = smem_u32(bars), empty = full + 8 * kStages, done = empty + 8 * kStages, freed = done + 16;

    if (threadIdx.x == 0) {
        s_quit = 0;
        for (int i = 0; i < kStages; ++i) {
            bar_init(full + 8 * i, 1);
            bar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(done + 8 * i, 1);
            bar_init(freed + 8 * i, 128);
        }
        bar_init_fence();
        prefetch_map(&map_a);
        prefetch_map(&map_b);
    }
    if (warp == 1) tmem_alloc(smem_u32(&s_tmem), 2 * BN);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    pdl_enter();

    const uint32_t nk = (p.depth + kBlockK - 1) / kBlockK;
    auto place = [&](uint32_t t, uint32_t& b, uint32_t& tm, uint32_t& tn) {
        b = t / p.tiles;
        t -= b * p.tiles;
        if (SYM) {
            triangle(t, tm, tn);
        } else {
            tm = t / p.tiles_n;
            tn = t - tm * p.tiles_n;
        }
    };

    if (warp == 0 && lane == 0) {
        uint32_t it = 0;   // fills so far
        bool ok = true;
        for (uint32_t t = blockIdx.x; t < p.total && ok; t += gridDim.x) {
            uint32_t b, tm, tn;
            place(t, b, tm, tn);
            for (uint32_t kb = 0; kb < nk; ++kb, ++it) {
                const uint32_t s = it % kStages;
                if (it >= kStages && !bar_wait(empty + 8 * s, (it / kStages - 1) & 1, quit)) {
                    ok = false;
                    break;
                }
                const uint32_t bar = full + 8 * s, sa = ring + s * kStageBytes, sb = sa + kABytes;
                const int k0 = static_cast<int>(kb * kBlockK);
                bar_expect(bar, kStageBytes);
                if (A_MN) {
#pragma unroll
                    for (int i = 0; i < kBlockM / 64; ++i)
                        copy_box(sa + i * 8192, &map_a, static_cast<int>(tm * kBlockM) + 64 * i, k0, static_cast<int>(b), bar);
                } else {
                    copy_box(sa, &map_a, k0, static_cast<int>(tm * kBlockM), static_cast<int>(b), bar);
                }
                if (B_MN) {
#pragma unroll
                    for (int i = 0; i < BN / 64; ++i)
                        copy_box(sb + i * 8192, &map_b, static_cast<int>(tn * BN) + 64 * i, k0, static_cast<int>(b), bar);
                } else {
#pragma unroll
                    for (int i = 0; i < BN / 128; ++i)
                        copy_box(sb + i * 16384, &map_b, k0, static_cast<int>(tn * BN) + 128 * i, static_cast<int>(b), bar);
                }
            }
        }
        if (!ok)   // the block must not leave with copies in flight
            for (uint32_t i = it > kStages ? it - kStages : 0; i < it; ++i)
                bar_drain(full + 8 * (i % kStages), (i / kStages) & 1);
    } else if (warp == 1 && lane == 0) {
        // fp32 accumulation, fp16 operands, 128 x BN
        constexpr uint32_t idesc = (1u << 4) | (A_MN ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u) |
                                   (static_cast<uint32_t>(BN >> 3) << 17) | (static_cast<uint32_t>(kBlockM >> 4) << 24);
        constexpr uint32_t step_a = (A_MN ? 2048u : 32u) >> 4, step_b = (B_MN ? 2048u : 32u) >> 4;
        uint32_t it = 0, n = 0;
        bool ok = true;
        for (uint32_t t = blockIdx.x; t < p.total && ok; t += gridDim.x, ++n) {
            const uint32_t acc = n & 1, d = tmem + acc * BN;
            if (n >= 2 && !bar_wait(freed + 8 * acc, (n / 2 - 1) & 1, quit)) break;
            tc_fence_after();
            for (uint32_t kb = 0; kb < nk; ++kb, ++it) {
                const uint32_t s = it % kStages;
                if (!bar_wait(full + 8 * s, (it / kStages) & 1, quit)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t sa = ring + s * kStageBytes;
                const uint64_t da = operand_desc(sa, 8192), db = operand_desc(sa + kABytes, 8192);
#pragma unroll
                for (int k = 0; k < kBlockK / 16; ++k)
                    mma_f16(d, da + k * step_a, db + k * step_b, idesc, kb > 0 || k > 0);
                tc_commit(empty + 8 * s);
            }
            if (ok) tc_commit(done + 8 * acc);
        }
        if (*quit) {   // nor free tensor memory under a product
            // a ring slot's barrier may be mid-phase, so finish on one of its own
            __shared__ __align__(8) uint64_t s_last;
            bar_init(smem_u32(&s_last), 1);
            bar_init_fence();
            tc_commit(smem_u32(&s_last));
            bar_drain(smem_u32(&s_last), 0);
        }
    } else if (warp >= 2) {
        const uint32_t quarter = warp & 3;
        uint32_t n = 0;
        for (uint32_t t = blockIdx.x; t < p.total; t += gridDim.x, ++n) {
            const uint32_t acc = n & 1;
            uint32_t b, tm, tn;
            place(t, b, tm, tn);
            const bool ok = bar_wait(done + 8 * acc, (n / 2) & 1, quit);
            if (__any_sync(0xFFFFFFFFu, !ok)) break;
            tc_fence_after();
            const uint32_t row = tm * kBlockM + quarter * 32 + lane;
            float f = p.f_acc;
            if (p.g0) {
                const float g = __ldg(p.g0 + b);
                f *= p.g_power == 2 ? g * g : g;
            }
            const uint64_t at = b * p.stride + static_cast<uint64_t>(row) * p.pitch;
#pragma unroll 1
            for (int cc = 0; cc < BN / 32; ++cc) {
                const uint32_t col = tn * BN + cc * 32;
                if (col >= p.cols) break;   // uniform over the warp
                float v[32];
                tmem_load32(tmem + acc * BN + cc * 32 + (quarter << 21), v);
                if (EPI == kPoly) {
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        uint4 x = make_uint4(0, 0, 0, 0);
                        if (row < p.rows && col + 8 * g < p.cols)
                            x = *reinterpret_cast<const uint4*>(p.lin + at + col + 8 * g);
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float l = widen<kFp16>((w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
                            float y = __fmaf_rn(v[8 * g + e], f, l * p.f_lin);
                            if (row == col + 8 * g + e) y += p.f_diag;
                            v[8 * g + e] = y;
                        }
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] *= f;
                }
                if (EPI == kFinal) {
                    if (row < p.rows) {
                        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.dst[b]) + static_cast<uint64_t>(row) * p.dst_ld;
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            const uint32_t c = col + 8 * g;
                            if (p.dst_vec && c + 8 <= p.cols) {
                                *reinterpret_cast<uint4*>(out + c) =
                                    make_uint4(pack_bf2(v[8 * g], v[8 * g + 1]), pack_bf2(v[8 * g + 2], v[8 * g + 3]),
                                               pack_bf2(v[8 * g + 4], v[8 * g + 5]), pack_bf2(v[8 * g + 6], v[8 * g + 7]));
                            } else {
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    if (c + e < p.cols) out[c + e] = __float2bfloat16_rn(v[8 * g + e]);
                            }
                        }
                    }
                } else {
                    if (row < p.rows) {
#pragma unroll
                        for (int g = 0; g < 4; ++g)
                            if (col + 8 * g < p.cols)   // whole vectors: the pitch is a multiple of 8
                                *reinterpret_cast<uint4*>(p.out + at + col + 8 * g) = make_uint4(
                                    pack_half2(v[8 * g], v[8 * g + 1]), pack_half2(v[8 * g + 2], v[8 * g + 3]),
                                    pack_half2(v[8 * g + 4], v[8 * g + 5]), pack_half2(v[8 * g + 6], v[8 * g + 7]));
                    }
                    if (SYM && tm != tn && row < p.rows) {
                        __half* mirror = p.out + b * p.stride + static_cast<uint64_t>(col) * p.pitch + row;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (col + e < p.cols) mirror[static_cast<uint64_t>(e) * p.pitch] = __float2half_rn(v[e]);
                    }
                }
            }
            tc_fence_before();
            bar_arrive(freed + 8 * acc);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_free(tmem, 2 * BN);
    }
}

// -------------------------------------------------------------------- host
// The scratch of a call, as offsets from its start.
struct Scratch {
    uint64_t partial, g0, x[2], s[3], bytes;
};
Scratch scratch_of(uint64_t batch, uint64_t rows, uint64_t cols) {
    const uint64_t side = rows < cols ? rows : cols;
    Scratch z;
    uint64_t at = 0;
    auto take = [&](uint64_t bytes) {
        const uint64_t here = at;
        at = up(at + bytes, 1024);
        return here;
    };
    z.partial = take(batch * kPartials * sizeof(double));
    z.g0 = take(batch * sizeof(float));
    for (uint64_t& x : z.x) x = take(batch * rows * up(cols, 8) * 2);
    for (uint64_t& s : z.s) s = take(batch * side * up(side, 8) * 2);
    z.bytes = at;
    return z;
}

template <int BN, bool A_MN, bool B_MN, int EPI, bool SYM>
cudaError_t product(int sms, const CUtensorMap& ma, const CUtensorMap& mb, ProductArgs& p, uint32_t batch,
                    cudaStream_t s) {
    const uint32_t tm = (p.rows + kBlockM - 1) / kBlockM;
    p.tiles_n = (p.cols + BN - 1) / BN;
    p.tiles = SYM ? tm * (tm + 1) / 2 : tm * p.tiles_n;
    p.total = p.tiles * batch;
    static_assert(!SYM || BN == kBlockM, "symmetric products take square tiles");
    constexpr auto kernel = k_ortho_product<BN, A_MN, B_MN, EPI, SYM>;
    const cudaError_t e = allow_smem<kernel>(product_smem(BN));
    if (e != cudaSuccess) return e;
    const unsigned grid = p.total < static_cast<uint32_t>(sms) ? p.total : static_cast<unsigned>(sms);
    return launch_pdl(kernel, dim3(grid), kProductThreads, product_smem(BN), 1, s, ma, mb, p);
}

// The update X <- p X (wide) or X p (tall), into scratch or the caller's matrices.
template <int EPI>
cudaError_t update(int sms, bool tall, const CUtensorMap& poly, const CUtensorMap& x_rows, const CUtensorMap& x_cols,
                   ProductArgs& p, uint32_t batch, cudaStream_t s) {
    return tall ? product<128, false, false, EPI, false>(sms, x_rows, poly, p, batch, s)
                : product<128, false, true, EPI, false>(sms, poly, x_cols, p, batch, s);
}

constexpr float kDefaultCoeffs[3] = {3.4445f, -4.7750f, 2.0315f};

}  // namespace

cudaError_t ortho_gave_up(cudaStream_t s, int32_t* out) { return read_gave_up(s, out); }

}  // namespace zg

using namespace zg;

extern "C" {

uint64_t zero_orthogonalize_workspace_bytes(int batch, uint64_t rows, uint64_t cols) {
    if (batch < 1 || batch > ZERO_MAX_MATRICES || rows < 1 || cols < 1 || rows > ZERO_MAX_SIDE || cols > ZERO_MAX_SIDE)
        return 0;
    return scratch_of(static_cast<uint64_t>(batch), rows, cols).bytes;
}

int zero_orthogonalize(int dtype, int batch, uint64_t rows, uint64_t cols, const void* const* src, uint64_t ld_src,
                       void* const* dst, uint64_t ld_dst, int steps, const float* coeffs, float scale, void* workspace,
                       uint64_t workspace_bytes, void* stream) {
    nvtxRangePushA("zero_orthogonalize");
    struct Pop { ~Pop() { nvtxRangePop(); } } pop;
    if (dtype != ZERO_FP16 && dtype != ZERO_BF16) return refuse(ZERO_EINVAL, "dtype must be fp16 or bf16");
    if (batch < 0 || batch > ZERO_MAX_MATRICES) return refuse(ZERO_EINVAL, "batch must be in 0..128");
    if (rows > ZERO_MAX_SIDE || cols > ZERO_MAX_SIDE) return refuse(ZERO_EINVAL, "a side is longer than ZERO_MAX_SIDE");
    if (steps < 1 || steps > ZERO_MAX_NS_STEPS) return refuse(ZERO_EINVAL, "steps must be in 1..32");
    if (!std::isfinite(scale)) return refuse(ZERO_EINVAL, "scale must be finite");
    if (coeffs)
        for (int i = 0; i < 3 * steps; ++i)
            if (!std::isfinite(coeffs[i])) return refuse(ZERO_EINVAL, "coeffs must be finite");
    if (batch == 0 || rows == 0 || cols == 0) return ZERO_OK;
    if (ld_src < cols || ld_dst < cols) return refuse(ZERO_EINVAL, "ld_src and ld_dst must be at least cols");
    if (ld_src > (1ull << 40) || ld_dst > (1ull << 40)) return refuse(ZERO_EINVAL, "ld_src or ld_dst too large");
    if (!src || !dst) return refuse(ZERO_EINVAL, "src or dst is NULL");
    const Scratch z = scratch_of(static_cast<uint64_t>(batch), rows, cols);
    if (!workspace || !aligned(workspace, 256)) return refuse(ZERO_EINVAL, "workspace is NULL or not 256-byte aligned");
    if (workspace_bytes < z.bytes)
        return refuse(ZERO_EINVAL, "workspace holds " + std::to_string(workspace_bytes) + " bytes, " +
                                       std::to_string(z.bytes) + " are needed");
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    const bool tall = rows > cols;
    const uint64_t side = tall ? cols : rows, span = tall ? rows : cols;
    const uint64_t xp = up(cols, 8), sp = up(side, 8);
    const uint32_t nb = static_cast<uint32_t>(batch);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);

    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return cuda_refuse(e, "zero_orthogonalize");

    PackArgs q = {};
    ProductArgs last = {};
    q.vec = ld_src % 8 == 0;
    last.dst_vec = ld_dst % 8 == 0;
    for (int i = 0; i < batch; ++i) {
        if (!src[i] || !aligned(src[i], 2)) return refuse(ZERO_EINVAL, "src[i] is NULL or not 2-byte aligned");
        if (!dst[i] || !aligned(dst[i], 2)) return refuse(ZERO_EINVAL, "dst[i] is NULL or not 2-byte aligned");
        q.src[i] = src[i];
        last.dst[i] = dst[i];
        q.vec &= aligned(src[i], 16);
        last.dst_vec &= aligned(dst[i], 16);
    }
    last.dst_ld = ld_dst;
    q.rows = rows;
    q.cols = cols;
    q.ld = ld_src;
    q.pitch = xp;
    q.segments = (cols + kSegment - 1) / kSegment;
    q.units = rows * q.segments;
    q.partial = reinterpret_cast<double*>(ws + z.partial);
    q.g0 = reinterpret_cast<float*>(ws + z.g0);
    q.x0 = reinterpret_cast<__half*>(ws + z.x[0]);
    const uint64_t want = (q.units + kPackWarps - 1) / kPackWarps;
    q.partials = static_cast<int>(want < kPartials ? want : kPartials);
    {
        const dim3 grid(static_cast<unsigned>(q.partials), nb);
        const dim3 packs(static_cast<unsigned>(want < 4096 ? want : 4096), nb);
        e = dtype == ZERO_FP16 ? launch_pdl(k_ortho_norm<kFp16>, grid, kThreads, 0, 1, s, q)
                               : launch_pdl(k_ortho_norm<kBf16>, grid, kThreads, 0, 1, s, q);
        if (e != cudaSuccess) return cuda_refuse(e, "norm");
        e = dtype == ZERO_FP16 ? launch_pdl(k_ortho_pack<kFp16>, packs, kThreads, 0, 1, s, q)
                               : launch_pdl(k_ortho_pack<kBf16>, packs, kThreads, 0, 1, s, q);
        if (e != cudaSuccess) return cuda_refuse(e, "pack");
    }

    // tensor maps: X by rows (K-major over columns, or MN-major blocks), the square ones by rows
    CUtensorMap x_k[2], x_mn[2], sq[3];
    for (int i = 0; i < 2; ++i) {
        const void* base = ws + z.x[i];
        if ((e = make_map(&x_k[i], 2, base, cols, rows, nb, xp, rows * xp, 64, 128)) != cudaSuccess ||
            (e = make_map(&x_mn[i], 2, base, cols, rows, nb, xp, rows * xp, 64, 64)) != cudaSuccess)
            return cuda_refuse(e, "tensor map");
    }
    for (int i = 0; i < 3; ++i)
        if ((e = make_map(&sq[i], 2, ws + z.s[i], side, side, nb, sp, side * sp, 64, 128)) != cudaSuccess)
            return cuda_refuse(e, "tensor map");

    auto square = [&](int to, uint64_t depth) {   // a symmetric product into square matrix `to`
        ProductArgs p = {};
        p.rows = p.cols = static_cast<uint32_t>(side);
        p.depth = static_cast<uint32_t>(depth);
        p.out = reinterpret_cast<__half*>(ws + z.s[to]);
        p.pitch = static_cast<uint32_t>(sp);
        p.stride = side * sp;
        return p;
    };
    // A = X X^T or X^T X of X buffer `x` into `to`; `raw`: that buffer still holds X0
    auto gram = [&](int to, int x, bool raw) {
        ProductArgs p = square(to, span);
        p.f_acc = raw ? kScaleA : kScaleA / (kScaleX * kScaleX);
        p.g0 = raw ? q.g0 : nullptr;
        p.g_power = 2;
        return tall ? product<128, true, true, kScale, true>(sms, x_mn[x], x_mn[x], p, nb, s)
                    : product<128, false, false, kScale, true>(sms, x_k[x], x_k[x], p, nb, s);
    };
    // to = a I + b A + c A^2
    auto poly = [&](int to, int a, const float* c) {
        ProductArgs p = square(to, side);
        p.lin = reinterpret_cast<const __half*>(ws + z.s[a]);
        p.f_diag = c[0] * kScaleB;
        p.f_lin = c[1] * (kScaleB / kScaleA);
        p.f_acc = c[2] * (kScaleB / (kScaleA * kScaleA));
        return product<128, false, false, kPoly, true>(sms, sq[a], sq[a], p, nb, s);
    };
    // to = B M, two commuting symmetric matrices, one of them of scale kScaleB
    auto commuting = [&](int to, int b, int m) {
        ProductArgs p = square(to, side);
        p.f_acc = 1.0f / kScaleB;
        return product<128, false, false, kScale, true>(sms, sq[b], sq[m], p, nb, s);
    };
    auto apply = [&](int x, int b, bool raw, bool to_dst) {
        ProductArgs p = last;
        p.rows = static_cast<uint32_t>(rows);
        p.cols = static_cast<uint32_t>(cols);
        p.depth = static_cast<uint32_t>(side);
        p.out = reinterpret_cast<__half*>(ws + z.x[x ^ 1]);
        p.pitch = static_cast<uint32_t>(xp);
        p.stride = rows * xp;
        p.g0 = raw ? q.g0 : nullptr;
        p.g_power = 1;
        if (to_dst) {
            p.f_acc = raw ? scale / kScaleB : scale / (kScaleB * kScaleX);
            return update<kFinal>(sms, tall, sq[b], x_k[x], x_mn[x], p, nb, s);
        }
        p.f_acc = raw ? kScaleX / kScaleB : 1.0f / kScaleB;
        return update<kScale>(sms, tall, sq[b], x_k[x], x_mn[x], p, nb, s);
    };

    int x = 0;
    for (int k = 0; k < steps;) {
        const float* c = coeffs ? coeffs + 3 * k : kDefaultCoeffs;
        const bool raw = k == 0, pair = raw && steps >= 2;
        if ((e = gram(0, x, raw)) != cudaSuccess || (e = poly(1, 0, c)) != cudaSuccess) return cuda_refuse(e, "product");
        int b = 1;
        if (pair) {
            const float* c1 = coeffs ? coeffs + 3 : kDefaultCoeffs;
            if ((e = commuting(2, 1, 0)) != cudaSuccess ||       // B A
                (e = commuting(0, 1, 2)) != cudaSuccess ||       // A_1 = B (B A)
                (e = poly(2, 0, c1)) != cudaSuccess ||           // B_1
                (e = commuting(0, 2, 1)) != cudaSuccess)         // Q = B_1 B
                return cuda_refuse(e, "product");
            b = 0;
        }
        k += pair ? 2 : 1;
        if ((e = apply(x, b, raw, k >= steps)) != cudaSuccess) return cuda_refuse(e, "product");
        x ^= 1;
    }
    return ZERO_OK;
}

}  // extern "C"
