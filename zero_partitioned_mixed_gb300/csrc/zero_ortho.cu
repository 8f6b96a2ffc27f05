// Newton-Schulz orthogonalisation of a batch of matrices (the update of the
// Muon optimiser) on the tensor cores.
//
//   X_0 = G / ||G||_F;   A = X X^T (over the shorter side);
//   X <- p(A) X,  p(A) = a I + b A + c A^2      (`steps` times)
//
// Precision.  Every stored matrix is fp16 times a fixed power of two (11 bits
// of significand against bf16's 8, at the same tensor rate); the products
// accumulate in fp32.  G itself is exact in that form, but for values 2^26
// times smaller than its largest.  The rounding that costs most is that of X
// while its small singular values are still small, so the first two steps do
// not form X_1 at all: with B = p(A) they compose A_1 = (B A) B and Q =
// p(A_1) B, and X_2 = Q X_0.  Against 64 bits a result before its rounding to
// bf16 is off by 1.0e-3 to 1.9e-3 (2-norm; gradients of low rank over noise,
// 64 x 64 to 768 x 2048), about what that rounding costs (1.7e-3); rounding
// every X gives up to 3.2e-3, and bf16 throughout 1e-2 to 2.5e-2.  That is the
// price against intermediates of 32 bits, which would leave the 1.7e-3 alone:
// with the rounding, measured on 6 to 24 matrices a size, 1.9e-3 to 2.2e-3 for
// shorter sides from 64 up, up to 3.3e-3 for 16 to 48, and below 16, where few
// values average, 2e-3 to 5e-3 in the mean and single matrices up to 2e-2.
//
// Work.  All products but the last of a step are symmetric: only tiles on or
// below the diagonal are computed, and each is written twice.  With the
// shorter side s and the longer l, the first two steps cost s^2 l + 5 s^3 +
// 2 s^2 l floating-point operations and each further one s^2 l + s^3 +
// 2 s^2 l (an ordinary product of s x l by l x s costs 2 s^2 l).  X is never
// transposed: a tall matrix takes its Gram matrix from MN-major operands and
// is multiplied from the right, a wide one the other way around.
//
// Two kernels by size.  A shorter side of at most 128 (and a longer one of at
// most 8192) stays on chip: k_ortho_small, one launch, 21 us for 96 x 160.
// Anything else goes through global memory (in practice L2): two streams that
// scale and pack G, then k_ortho_products, all products in one cooperative
// launch.  Measured with five steps: 12 x 768 x 768 186 us, 6 x 1531 x 1003
// 249 us, 11008 x 4096 1.92 ms, which is 1.44 PFLOP/s of the operations above
// (75 % of a plain bf16 product's rate).

#include <cmath>
#include <cstdint>
#include <cstring>
#include <string>

#include <nvtx3/nvToolsExt.h>

#include "zero_gb300.h"
#include "zero_rows.cuh"
#include "zero_tc.cuh"

namespace zg {
namespace {

constexpr int kMaxMatrices = ZERO_MAX_MATRICES;

// After settle(): the step that the matrices are part of learns of a wait that
// gave up, before its zero_muon_apply runs.  `pending`: of its state, or NULL.
__device__ __forceinline__ void note_gave_up(volatile int* quit, int32_t* pending) {
    if (*quit && pending && threadIdx.x == 0) atomicOr(pending, ZERO_MUON_GAVE_UP);
}

constexpr int kMaxPhases = 3 * ZERO_MAX_NS_STEPS + 3;

// Storage scales (all powers of two): entries of X and A are at most a
// little over 1, those of p(A) and Q at most a^2 or so.
constexpr float kScaleX = 8192.0f, kScaleA = 4096.0f, kScaleB = 128.0f;

// ----------------------------------------------------- scaling and packing
// X0 = G 2^k in fp16, k such that the largest magnitude lies in [2^12, 2^13),
// and g0 = 1 / ||X0||, which the products that read X0 take into their scale.
// Scaled like that, squares and their sums stay in fp32's range whatever G's
// magnitudes are (a value whose square underflows is 2^-70 of the largest).
// One pass finds the largest magnitude, one packs and sums the squares; both
// are streams, the second mostly out of L2.  A matrix is read in units of
// kPackRows rows by 256 columns, one warp a unit, 8 values a lane and row,
// the rows' loads in flight together.
constexpr int kPackRows = 4;
constexpr int kPackWarps = kThreads / 32;
constexpr uint32_t kTopBlocks = 1024;   // blocks of the first pass for one matrix, at most

struct PackArgs {
    const void* src[kMaxMatrices];
    uint64_t rows, cols, ld, pitch;
    uint32_t segments, units;   // 256-column segments a row; units a matrix
    uint32_t tops, sums;        // blocks a matrix of the two passes
    uint32_t* top;              // [batch][kTopBlocks] largest magnitudes, as 16-bit patterns
    float* sum;                 // [batch][sums] sums of squares of X0
    uint32_t* ticket;           // [batch] finished blocks of the second pass
    float* g0;                  // [batch]
    uint32_t* done;             // [batch][kMaxPhases], cleared for the products
    __half* x0;                 // [batch][rows][pitch]
};

// A lane's values of unit `u`: row0 + r, columns c to c + 7, packed; zeros
// past the matrix.
__device__ __forceinline__ void load_unit(const PackArgs& a, int b, uint32_t u, uint64_t& row0, uint64_t& c,
                                          uint32_t (&w)[kPackRows][4]) {
    const uint32_t group = u / a.segments;
    c = (u - group * a.segments) * 256u + 8 * (threadIdx.x & 31);
    row0 = static_cast<uint64_t>(group) * kPackRows;
    const unsigned short* src = static_cast<const unsigned short*>(a.src[b]);
    const int64_t total = static_cast<int64_t>((a.rows - 1) * a.ld + a.cols);
#pragma unroll
    for (int r = 0; r < kPackRows; ++r) {
        if (row0 + r < a.rows) load8(src, static_cast<int64_t>((row0 + r) * a.ld + c), total, w[r]);
        else w[r][0] = w[r][1] = w[r][2] = w[r][3] = 0;
    }
    const int valid = values_left(a.cols, c);
#pragma unroll
    for (int r = 0; r < kPackRows; ++r) clear_from(w[r], valid);
}

// Block-wide results in every thread, in a fixed order.
__device__ __forceinline__ uint32_t block_top(uint32_t x) {
    __shared__ uint32_t s[32];
    x = __reduce_max_sync(0xFFFFFFFFu, x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0;
    for (uint32_t i = 0; i < blockDim.x / 32; ++i) x = max(x, s[i]);
    return x;
}
__device__ __forceinline__ float block_sum32(float x) {
    __shared__ float s[32];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, off);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0.0f;
    for (uint32_t i = 0; i < blockDim.x / 32; ++i) x += s[i];
    return x;
}

// The two factors of 2^k (each a normal fp32 number) from the largest
// magnitude's pattern; 1 for a zero matrix.  An infinity or a NaN stays one.
template <int DT>
__device__ __forceinline__ void scale_factors(uint32_t top, float& m0, float& m1) {
    const float x = widen<DT>(top);
    const int e = x > 0.0f && x < INFINITY ? 12 - ilogbf(x) : 0;
    m0 = ldexpf(1.0f, e / 2);
    m1 = ldexpf(1.0f, e - e / 2);
}
// g0 from the sum of squares of X0: 0 for a zero matrix, NaN where G has an
// infinity or a NaN.
__device__ __forceinline__ float inverse_norm(float sum, uint32_t top, uint32_t infinite) {
    return top >= infinite ? NAN : top == 0u ? 0.0f : 1.0f / sqrtf(sum);
}
template <int DT>
__device__ constexpr uint32_t infinity_pattern() { return DT == kBf16 ? 0x7F80u : 0x7C00u; }

// 8 packed values times m0 m1 in fp16; adds their squares to `sum`.
template <int DT>
__device__ __forceinline__ void scale8(const uint32_t (&w)[4], float m0, float m1, uint32_t (&q)[4], float& sum) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float lo, hi;
        widen2<DT>(w[e], lo, hi);
        mul2(lo, hi, m0);
        mul2(lo, hi, m1);
        sum = __fmaf_rn(hi, hi, __fmaf_rn(lo, lo, sum));
        q[e] = narrow2<kFp16>(lo, hi);
    }
}

__global__ void __launch_bounds__(kThreads) k_ortho_top(const __grid_constant__ PackArgs a) {
    pdl_enter();
    const int b = blockIdx.y;
    if (blockIdx.x == 0) {
        for (int i = threadIdx.x; i < kMaxPhases; i += kThreads) a.done[static_cast<uint64_t>(b) * kMaxPhases + i] = 0u;
        if (threadIdx.x == 0) a.ticket[b] = 0u;
    }
    uint32_t top = 0;
    for (uint32_t u = blockIdx.x * kPackWarps + (threadIdx.x >> 5); u < a.units; u += gridDim.x * kPackWarps) {
        uint64_t row0, c;
        uint32_t w[kPackRows][4];
        load_unit(a, b, u, row0, c, w);
#pragma unroll
        for (int r = 0; r < kPackRows; ++r) top = max(top, top_pattern(w[r]));
    }
    top = block_top(top);
    if (threadIdx.x == 0) a.top[static_cast<uint64_t>(b) * kTopBlocks + blockIdx.x] = top;
}

// One unit a warp, its loads in flight while the scale is put together; the
// last block of a matrix adds up the sums.
template <int DT>
__global__ void __launch_bounds__(kThreads) k_ortho_pack(const __grid_constant__ PackArgs a) {
    pdl_enter();
    __shared__ int s_last;
    const int b = blockIdx.y;
    const uint32_t u = blockIdx.x * kPackWarps + (threadIdx.x >> 5);
    uint64_t row0 = a.rows, c = a.cols;
    uint32_t w[kPackRows][4] = {};
    if (u < a.units) load_unit(a, b, u, row0, c, w);
    uint32_t top = 0;
    for (uint32_t i = threadIdx.x; i < a.tops; i += kThreads) top = max(top, a.top[static_cast<uint64_t>(b) * kTopBlocks + i]);
    top = block_top(top);
    float m0, m1, sum = 0.0f;
    scale_factors<DT>(top, m0, m1);
    if (c < a.cols) {
        __half* out = a.x0 + (static_cast<uint64_t>(b) * a.rows + row0) * a.pitch + c;
#pragma unroll
        for (int r = 0; r < kPackRows; ++r, out += a.pitch) {
            if (row0 + r >= a.rows) break;
            uint32_t q[4];
            scale8<DT>(w[r], m0, m1, q, sum);
            // whole eights: the pitch is a multiple of 8
            *reinterpret_cast<uint4*>(out) = make_uint4(q[0], q[1], q[2], q[3]);
        }
    }
    sum = block_sum32(sum);
    if (threadIdx.x == 0) {
        a.sum[static_cast<uint64_t>(b) * a.sums + blockIdx.x] = sum;
        __threadfence();
        s_last = atomicAdd(&a.ticket[b], 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    sum = 0.0f;
    for (uint32_t i = threadIdx.x; i < a.sums; i += kThreads) sum += __ldcg(a.sum + static_cast<uint64_t>(b) * a.sums + i);
    sum = block_sum32(sum);
    if (threadIdx.x == 0) a.g0[b] = inverse_norm(sum, top, infinity_pattern<DT>());
}

// ---------------------------------------------------------------- products
// All products of a call run in one kernel.  Each is a phase: for every
// matrix of the batch, out = epilogue(A B^T), A having the output's rows and
// B its columns, both over `depth`.  A tile of a phase waits until the
// matrix's previous phase is complete (a counter per matrix and phase), so
// the matrices of a batch run through the phases independently, without a
// launch or a grid-wide barrier between them.  Tiles are handed out in
// order of phase, matrix, tile, round robin over the CTA pairs, so every
// tile depends on earlier ones only, and the launch is cooperative: every
// wait ends.  For small matrices the chain of sixteen phases bounds it, some
// 10 us each: an input's way from L2 1 us, the products 3 us (768 values),
// their end 1 us, the epilogue 2 us, its stores and the counter 1.3 us, the
// next phase's sight of it 1.3 us.  Large ones lose most to whole rounds of
// tiles (136 tiles of 4096 x 4096 on 76 pairs take two).
enum Epi : int32_t {
    kScale,   // out = f acc
    kPoly,    // out = f acc + f_lin lin + f_diag I
    kFinal,   // bf16, into the caller's matrices: out = f acc
};

struct Phase {
    int32_t a, b;              // tensor maps of the operands
    int32_t a_mn, b_mn;        // their order in memory: 0 K-major, 1 MN-major
    int32_t out;               // tensor map of the output
    int32_t symmetric;         // tiles on and below the diagonal, each written with its mirror image
    int32_t lin;               // tensor map of the linear term
    Epi epi;
    uint32_t rows, cols, depth;
    uint32_t tiles_n, tiles;   // tiles a row, a matrix
    float f_acc, f_lin, f_diag;
    int32_t g_power;           // further factor g0[b]^g_power
};

enum Map : int { kXRows0, kXRows1, kXCols0, kXCols1, kSquare0, kSquare1, kSquare2,   // operands
                 kXOut0, kXOut1, kSquareOut0, kSquareOut1, kSquareOut2, kMaps };    // outputs (and linear terms)

struct ProductArgs {
    CUtensorMap maps[kMaps];
    Phase phases[kMaxPhases];
    void* dst[kMaxMatrices];   // kFinal
    uint64_t dst_ld;
    const float* g0;           // [batch]
    uint32_t* done;            // [batch][kMaxPhases] finished epilogues, zero at the start
    int32_t* pending;          // of the step's state, or NULL
    int32_t dst_vec;           // every row of dst starts on 16 bytes
    uint32_t n_phases, batch;
    uint32_t hold;             // zero_debug_hold_matrix, or 0
};

// A pair of CTAs computes 256 x 256 tiles: a stage of 64 steps of the
// contraction is 32 KiB a CTA for 512 cycles of products, which is about
// what an SM gets from L2 (128 x 128 tiles of one CTA need twice that, and
// ran at 0.9 PFLOP/s, 2.85 ms for 11008 x 4096).  Warp 0 copies operands into a ring of stages, warp 1
// of the leader issues the products, warps 2 to 9 turn finished accumulators
// into output (each 32 rows by 128 columns of a tile, by 32 columns at a
// time); two accumulators in tensor memory, so that one tile's epilogue runs
// under the next one's products.  Between dependent phases an epilogue is not
// hidden: eight warps take 2 us where four took 4 (8 with a linear term).
constexpr int kTile = 256, kHalf = 128, kBlockK = 64;
constexpr int kOutWarps = 8, kProductThreads = 64 + 32 * kOutWarps;
constexpr int kStages = 5;
constexpr uint32_t kOperandBytes = kHalf * kBlockK * 2, kStageBytes = 2 * kOperandBytes;
// A warp's output buffers: 32 x 32 values twice, and twice their mirror image.
constexpr uint32_t kOutBytes = 32 * 32 * 2, kWarpBytes = 4 * kOutBytes;
constexpr size_t kProductSmem = 1024 + kStages * kStageBytes + kOutWarps * kWarpBytes;
static_assert(kProductSmem >= kAloneSmem, "see tmem_alloc");
constexpr uint32_t kDonePerTile = 2 * kOutWarps;   // the warps of 2 CTAs

// The tiles of one CTA pair, in order.
struct Walk {
    const ProductArgs& p;
    uint32_t phase, at;   // `at`: index within the phase
    uint32_t b, tm, tn;
    __device__ explicit Walk(const ProductArgs& args) : p(args), phase(0), at(blockIdx.x >> 1), b(0), tm(0), tn(0) {}
    __device__ bool find() {
        while (phase < p.n_phases) {
            const Phase& f = p.phases[phase];
            const uint32_t total = f.tiles * p.batch;
            if (at < total) {
                b = at / f.tiles;
                const uint32_t t = at - b * f.tiles;
                if (f.symmetric) {
                    triangle(t, tm, tn);
                } else {
                    tm = t / f.tiles_n;
                    tn = t - tm * f.tiles_n;
                }
                return true;
            }
            at -= total;
            ++phase;
        }
        return false;
    }
    __device__ bool next() {
        at += gridDim.x >> 1;
        return find();
    }
    // Waits for the matrix's previous phase.
    __device__ bool inputs_ready(volatile int* quit) const {
        if (phase == 0) return true;
        return count_wait(p.done + static_cast<uint64_t>(b) * kMaxPhases + phase - 1,
                          p.phases[phase - 1].tiles * kDonePerTile, quit);
    }
};

__global__ void __launch_bounds__(kProductThreads) k_ortho_products(const __grid_constant__ ProductArgs p) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * kStages + 4 + kOutWarps];
    __shared__ __align__(8) uint64_t s_last;
    __shared__ uint32_t s_tmem;
    __shared__ int s_quit;
    volatile int* quit = &s_quit;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t full = smem_u32(bars), empty = full + 8 * kStages, done = empty + 8 * kStages, freed = done + 16,
                   lin0 = freed + 16;
    if (threadIdx.x == 0) {
        s_quit = 0;
        const int held = blockIdx.x == 0 ? static_cast<int>(p.hold) : 0;
        for (int i = 0; i < kStages; ++i) {
            bar_init(full + 8 * i, i + 1 == held ? 2 : 1);
            bar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(done + 8 * i, 1);
            bar_init(freed + 8 * i, 2 * kOutWarps);
        }
        for (int i = 0; i < kOutWarps; ++i) bar_init(lin0 + 8 * i, 1);
        bar_init(smem_u32(&s_last), 1);
        bar_init_fence();
    }
    if (warp == 1) tmem_alloc_pair(smem_u32(&s_tmem), 2 * kTile);
    {   // the phases into the constant cache: a first read there costs microseconds
        uint32_t touched = 0;
        for (uint32_t i = 0; i < p.n_phases; ++i) touched |= p.phases[i].tiles;
        if (touched == 0u) s_quit = 0;   // never; keeps the reads
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = s_tmem;

    if (warp == 0 && elect_one()) {
        const uint32_t leader_full = cluster_addr(full, 0);
        Ring<kStages> r;
        bool ok = true;
        Walk w(p);
        for (bool more = w.find(); more && ok; more = w.next()) {
            const Phase& f = p.phases[w.phase];
            if (!w.inputs_ready(quit)) break;
            proxy_fence_global();
            const uint32_t nk = (f.depth + kBlockK - 1) / kBlockK;
            const CUtensorMap *ma = &p.maps[f.a], *mb = &p.maps[f.b];
            const int ra = static_cast<int>(w.tm * kTile + rank * kHalf);
            const int rb = static_cast<int>(w.tn * kTile + rank * kHalf), z = static_cast<int>(w.b);
            const bool a_mn = f.a_mn, b_mn = f.b_mn;
            for (uint32_t kb = 0; kb < nk; ++kb, r.next()) {
                if (!bar_wait(empty + 8 * r.s, r.parity ^ 1, quit, kForSpace)) {   // passes at once in the first round
                    ok = false;
                    break;
                }
                const uint32_t bar = leader_full + 8 * r.s, sa = ring + r.s * kStageBytes, sb = sa + kOperandBytes;
                const int k0 = static_cast<int>(kb * kBlockK);
                if (rank == 0) bar_expect(full + 8 * r.s, 2 * kStageBytes);   // the bytes of both CTAs
                if (a_mn) {
                    copy_box_pair(sa, ma, ra, k0, z, bar);
                    copy_box_pair(sa + 8192, ma, ra + 64, k0, z, bar);
                } else {
                    copy_box_pair(sa, ma, k0, ra, z, bar);
                }
                if (b_mn) {
                    copy_box_pair(sb, mb, rb, k0, z, bar);
                    copy_box_pair(sb + 8192, mb, rb + 64, k0, z, bar);
                } else {
                    copy_box_pair(sb, mb, k0, rb, z, bar);
                }
            }
        }
    } else if (warp == 1 && rank == 0 && elect_one()) {
        const uint64_t desc0 = operand_desc(ring, 8192);
        Ring<kStages> r;
        uint32_t n = 0;
        bool ok = true;
        Walk w(p);
        for (bool more = w.find(); more && ok; more = w.next(), ++n) {
            const Phase& f = p.phases[w.phase];
            // fp32 accumulation, fp16 operands, 256 x 256
            const uint32_t idesc = (1u << 4) | (f.a_mn ? 1u << 15 : 0u) | (f.b_mn ? 1u << 16 : 0u) |
                                   (static_cast<uint32_t>(kTile >> 3) << 17) | (static_cast<uint32_t>(kTile >> 4) << 24);
            const uint32_t step_a = (f.a_mn ? 2048u : 32u) >> 4, step_b = (f.b_mn ? 2048u : 32u) >> 4;
            const uint32_t acc = n & 1, d = tmem + acc * kTile;
            if (n >= 2 && !bar_wait(freed + 8 * acc, (n / 2 - 1) & 1, quit, kForSpace)) break;
            tc_fence_after();
            const uint32_t nk = (f.depth + kBlockK - 1) / kBlockK;
            for (uint32_t kb = 0; kb < nk; ++kb, r.next()) {
                if (!bar_wait(full + 8 * r.s, r.parity, quit, kForData)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t da = desc0 + r.s * (kStageBytes >> 4), db = da + (kOperandBytes >> 4);
#pragma unroll
                for (int k = 0; k < kBlockK / 16; ++k)
                    mma_f16_pair(d, da + k * step_a, db + k * step_b, idesc, kb > 0 || k > 0);
                tc_commit_pair(empty + 8 * r.s);
            }
            if (ok) tc_commit_pair(done + 8 * acc);
        }
        if (*quit) {   // tensor memory must not be freed under a product
            tc_commit_pair(smem_u32(&s_last));
            bar_drain(smem_u32(&s_last), 0, now_ns());
        }
    } else if (warp >= 2) {
        const uint32_t quarter = warp & 3;   // the lanes of tensor memory that this warp can read
        const uint32_t part = static_cast<uint32_t>(warp - 2) >> 2;   // its half of the columns
        const uint32_t mine = ring + kStages * kStageBytes + static_cast<uint32_t>(warp - 2) * kWarpBytes;
        const uint32_t leader_freed = cluster_addr(freed, 0), lin_bar = lin0 + 8 * static_cast<uint32_t>(warp - 2);
        uint32_t n = 0, lin_parity = 0;
        Walk w(p);
        for (bool more = w.find(); more; more = w.next(), ++n) {
            const Phase& f = p.phases[w.phase];
            const uint32_t acc = n & 1;
            const uint32_t row0 = w.tm * kTile + rank * kHalf + quarter * 32;
            const uint32_t col0 = w.tn * kTile + part * 128;
            const int z = static_cast<int>(w.b);
            const bool poly = f.epi == kPoly, final = f.epi == kFinal, mirror = f.symmetric && w.tm != w.tn;
            // chunks of 32 columns that hold output
            const uint32_t chunks = row0 >= f.rows || col0 >= f.cols ? 0u : min(4u, (f.cols - col0 + 31u) / 32u);
            bool ok = true;
            uint4 lin[4][4];   // this lane's row of the linear term, fetched under the products
            if (poly && chunks) {
                // through the output buffers, which are free: the last tile's stores were waited for
                if (lane == 0) {
                    ok = w.inputs_ready(quit);
                    if (ok) {
                        proxy_fence();
                        bar_expect(lin_bar, chunks * kOutBytes);
                        for (uint32_t c = 0; c < chunks; ++c)
                            copy_box(mine + c * kOutBytes, &p.maps[f.lin], static_cast<int>(col0 + 32 * c),
                                     static_cast<int>(row0), z, lin_bar);
                    }
                }
                ok = __all_sync(0xFFFFFFFFu, ok) && bar_wait(lin_bar, lin_parity, quit, kForData);
                lin_parity ^= 1;
#pragma unroll
                for (uint32_t c = 0; c < 4; ++c)
#pragma unroll
                    for (uint32_t j = 0; j < 4; ++j) lin[c][j] = ld_shared(mine + c * kOutBytes + piece64(lane, j));
            }
            ok = ok && bar_wait(done + 8 * acc, (n / 2) & 1, quit);
            if (__any_sync(0xFFFFFFFFu, !ok)) break;
            tc_fence_after();
            float scale = f.f_acc;
            if (f.g_power) {
                const float g = __ldg(p.g0 + w.b);
                scale *= f.g_power == 2 ? g * g : g;
            }
            const float f_lin = f.f_lin, f_diag = f.f_diag;
            const uint32_t acc0 = tmem + acc * kTile + part * 128 + (quarter << 21);
            uint32_t v[2][32];
            if (chunks) tmem_start32(acc0, v[0]);
#pragma unroll
            for (uint32_t c = 0; c < 4; ++c) {
                if (c >= chunks) break;
                uint32_t (&a)[32] = v[c & 1];
                tmem_wait(a);
                if (c + 1 < chunks) tmem_start32(acc0 + 32 * (c + 1), v[(c + 1) & 1]);
                const uint32_t buf = mine + (c & 1) * kOutBytes, flip = mine + (2 + (c & 1)) * kOutBytes;
                uint32_t q[16];
                if (poly) {
                    const uint32_t lw[16] = {lin[c][0].x, lin[c][0].y, lin[c][0].z, lin[c][0].w, lin[c][1].x, lin[c][1].y,
                                             lin[c][1].z, lin[c][1].w, lin[c][2].x, lin[c][2].y, lin[c][2].z, lin[c][2].w,
                                             lin[c][3].x, lin[c][3].y, lin[c][3].z, lin[c][3].w};
#pragma unroll
                    for (uint32_t e = 0; e < 16; ++e) {
                        float lo, hi;
                        widen2<kFp16>(lw[e], lo, hi);
                        a[2 * e] = __float_as_uint(__fmaf_rn(__uint_as_float(a[2 * e]), scale, lo * f_lin));
                        a[2 * e + 1] = __float_as_uint(__fmaf_rn(__uint_as_float(a[2 * e + 1]), scale, hi * f_lin));
                    }
                    if (row0 == col0 + 32 * c) {   // the diagonal's chunk
                        // f_diag is added as a value, zero or not: a test of each turns into a branch a lane
#pragma unroll
                        for (uint32_t e = 0; e < 32; ++e)
                            a[e] = __float_as_uint(__uint_as_float(a[e]) + (lane == e ? f_diag : 0.0f));
                    }
                } else {
#pragma unroll
                    for (uint32_t e = 0; e < 32; ++e) a[e] = __float_as_uint(__uint_as_float(a[e]) * scale);
                }
                if (final) {
#pragma unroll
                    for (uint32_t e = 0; e < 16; ++e) q[e] = narrow2<kBf16>(__uint_as_float(a[2 * e]), __uint_as_float(a[2 * e + 1]));
                } else {
#pragma unroll
                    for (uint32_t e = 0; e < 16; ++e) q[e] = narrow2<kFp16>(__uint_as_float(a[2 * e]), __uint_as_float(a[2 * e + 1]));
                }
                if (lane == 0) store_wait_read<1>();   // the stores of chunk c - 2 have left its buffers
                __syncwarp();
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j)
                    st_shared(buf + piece64(lane, j), q[4 * j], q[4 * j + 1], q[4 * j + 2], q[4 * j + 3]);
                if (mirror) {
                    // columns become rows: two lanes trade halves, the even one then holds column 2e of
                    // its own and the next row, the odd one column 2e + 1 of the previous and its own
#pragma unroll
                    for (uint32_t e = 0; e < 16; ++e) {
                        const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, q[e], 1);
                        const uint32_t word = lane & 1 ? __byte_perm(other, q[e], 0x7632) : __byte_perm(q[e], other, 0x5410);
                        st_shared(flip + piece64(2 * e + (lane & 1), lane >> 3) + 4 * ((lane >> 1) & 3), word);
                    }
                }
                if (final) {
                    __syncwarp();
                    write_rows(static_cast<unsigned short*>(p.dst[w.b]), p.dst_ld, p.dst_vec, f.rows, f.cols, row0,
                                   col0 + 32 * c, buf);
                } else {
                    proxy_fence_shared();
                    __syncwarp();
                    if (lane == 0) {
                        const int y = static_cast<int>(row0), x = static_cast<int>(col0 + 32 * c);
                        store_box(&p.maps[f.out], x, y, z, buf);
                        if (mirror) store_box(&p.maps[f.out], y, x, z, flip);
                        store_commit();
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                bar_arrive_cluster(leader_freed + 8 * acc);
                if (!final) {   // the tile's output is in memory before it counts
                    store_wait<0>();
                    proxy_fence_global();
                    count_done(p.done + static_cast<uint64_t>(w.b) * kMaxPhases + w.phase);
                }
            }
            __syncwarp();
        }
        if (lane == 0) store_wait<0>();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    settle(quit);
    note_gave_up(quit, p.pending);
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_free_pair(tmem, 2 * kTile);
    }
    __syncwarp();
    cluster_sync();
}

// ----------------------------------------------------- short sides up to 128
// A matrix whose shorter side is at most 128 stays on the SM: one CTA holds up
// to 512 of the longer side's values (fewer while there are SMs for that), a
// cluster of up to 8 CTAs the whole of it (16 for a longer side above 4096,
// where global memory took 231 us for 100 x 8192, not 59; and above 2048 while
// such clusters fit side by side: 128 x 4096 took 55 us in 8, 51 in 16), and
// the square matrices are computed by each CTA for itself.  Only X X^T is
// summed over the cluster, through its shared memory.  The sixteen dependent
// products of five steps take about a microsecond each this way; through
// global memory they took five.
// Bound by that chain and by the copies in and out, on few SMs.  Five steps of
// bf16: 96 x 160 21 us, 23 x 1519 28, 128 x 4096 49, 100 x 8192 58, 100
// matrices of 48 x 300 26, 60 of 100 x 2000 97.
//
// X lies as the caller has it, in blocks of 64 columns whose rows are 128
// bytes.  That one layout serves both products: of a wide matrix the blocks
// are K-major operands of X X^T and MN-major ones of B X, of a tall one
// MN-major operands of X^T X and K-major ones of X B.
//
// All of it runs once a launch, mostly out of a cold instruction cache, so the
// code is kept short: one copy of the products' code for all of them, and
// loads that need no registers (cp.async).
constexpr uint32_t kSide = 128, kSlabBlocks = 8, kMaxCtas = 16, kPortableCtas = 8;
constexpr uint32_t kBlockBytes = kSide * 128;   // half a square
constexpr uint32_t kSquareBytes = 2 * kBlockBytes;
constexpr uint32_t kSlabUnit = 64 * kSide * 2;  // bytes of X for 64 of the longer side
// 16 warps: a form in which 8 of them take the products' results took 61 us against 55 for 128 x 4096 and 30 against
// 26 for 128 x 256 (31 against 33 for 23 x 1519, whose results are smaller).
constexpr int kSmallThreads = 512;

struct SmallArgs {
    const void* src[kMaxMatrices];
    void* dst[kMaxMatrices];
    uint64_t ld_src, ld_dst;
    uint32_t side, span;     // the shorter and the longer side
    uint32_t ctas, per;      // CTAs a matrix, 64s of the longer side a CTA
    int32_t tall, steps;
    uint32_t arrivals;       // that a product's end takes: 1, or with zero_debug_hold_matrix one more, which never comes
    int32_t* pending;        // of the step's state, or NULL
    float scale;
    float coeffs[3 * ZERO_MAX_NS_STEPS];
};

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
    uint32_t x;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(addr) : "memory");
    return x;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t x, uint32_t y) {
    asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(x), "r"(y) : "memory");
}
// 16 bytes into shared memory, the last 16 - `bytes` of them zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

template <int DT>
__global__ void __launch_bounds__(kSmallThreads) k_ortho_small(const __grid_constant__ SmallArgs p) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t s_bar;
    __shared__ uint32_t s_tmem;
    __shared__ int s_quit;
    __shared__ uint32_t s_top;
    __shared__ float s_sum;
    __shared__ float s_coeffs[3 * ZERO_MAX_NS_STEPS];   // a first read of a parameter costs microseconds: not in between
    volatile int* quit = &s_quit;
    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = p.ctas > 1 ? cluster_rank() : 0, b = blockIdx.x / p.ctas;
    const uint32_t first = rank * p.per * 64;                       // this CTA's part of the longer side
    const uint32_t span = min(p.span - first, p.per * 64);
    const bool tall = p.tall;
    // 64s of it; an even number of a tall matrix, whose products take 128 rows at a time
    const uint32_t blocks = tall ? (span + 127) / 128 * 2 : (span + 63) / 64;
    const uint32_t block_bytes = tall ? blocks * 8192 : kBlockBytes;   // from 64 columns of X to the next
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t sq0 = base, x = base + 3 * kSquareBytes;         // three squares, then X
    const uint32_t bar = smem_u32(&s_bar);
    if (tid == 0) {
        s_quit = 0;
        bar_init(bar, p.arrivals);
        bar_init_fence();
    }
    if (warp == 0) tmem_alloc(smem_u32(&s_tmem), 512);
    __syncthreads();   // tensor memory is held before the next kernel may come (pdl_enter)
    pdl_enter();
    for (uint32_t i = tid; i < 3u * p.steps; i += kSmallThreads) s_coeffs[i] = p.coeffs[i];
    for (uint32_t i = tid; i < blocks * (kSlabUnit / 16); i += kSmallThreads) st_shared(x + 16 * i, 0u, 0u, 0u, 0u);
    if (p.ctas > 1)   // what the cluster's sums leave out
        for (uint32_t i = tid; i < kSquareBytes / 16; i += kSmallThreads) st_shared(sq0 + 16 * i, 0u, 0u, 0u, 0u);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;

    // G as it is into X, 16 bytes at a time where its rows start on 16 bytes
    const uint32_t rows = tall ? span : p.side, cols = tall ? p.side : span;
    auto place = [&](uint32_t r, uint32_t c) {
        return x + (c >> 6) * block_bytes + piece128(r, (c & 63) >> 3) + 2 * (c & 7);
    };
    const uint32_t eights = (cols + 7) / 8;
    {
        const unsigned short* src = static_cast<const unsigned short*>(p.src[b]) + (tall ? first * p.ld_src : first);
        if ((reinterpret_cast<uintptr_t>(src) & 15) == 0 && p.ld_src % 8 == 0) {
#pragma unroll 1
            for (uint32_t i = tid; i < rows * eights; i += kSmallThreads) {
                const uint32_t r = i / eights, c = (i - r * eights) * 8;
                copy16(place(r, c), src + r * p.ld_src + c, 2 * min(8u, cols - c));
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        } else {   // the aligned pieces that cover 8 values, for two eights at a time (3 x 7777 x 113: 83 us, by value 90)
            const unsigned short* from = static_cast<const unsigned short*>(p.src[b]);
            const int64_t total = static_cast<int64_t>(((tall ? p.span : p.side) - 1) * p.ld_src + (tall ? p.side : p.span));
            const uint64_t start = tall ? first * p.ld_src : first;
#pragma unroll 1
            for (uint32_t i0 = tid; i0 < rows * eights; i0 += 2 * kSmallThreads) {
                uint32_t w[2][4];
#pragma unroll
                for (uint32_t k = 0; k < 2; ++k) {
                    const uint32_t i = i0 + k * kSmallThreads, r = i / eights, c = (i - r * eights) * 8;
                    if (r < rows) load8(from, static_cast<int64_t>(start + r * p.ld_src + c), total, w[k]);
                }
#pragma unroll
                for (uint32_t k = 0; k < 2; ++k) {
                    const uint32_t i = i0 + k * kSmallThreads, r = i / eights, c = (i - r * eights) * 8;
                    if (r >= rows) continue;
                    clear_from(w[k], static_cast<int>(cols - c));
                    st_shared(place(r, c), w[k][0], w[k][1], w[k][2], w[k][3]);
                }
            }
        }
    }
    __syncthreads();
    // its largest magnitude
    uint32_t top = 0;
#pragma unroll 2
    for (uint32_t i = tid; i < blocks * (kSlabUnit / 16); i += kSmallThreads) {
        const uint4 v = ld_shared(x + 16 * i);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        top = max(top, top_pattern(w));
    }
    top = block_top(top);
    if (p.ctas > 1) {
        if (tid == 0) s_top = top;
        cluster_sync();
        for (uint32_t q = 0; q < p.ctas; ++q) top = max(top, ld_cluster_u32(cluster_addr(smem_u32(&s_top), q)));
    }
    // X0 = G 2^k in place, and its sum of squares
    float m0, m1, sum = 0.0f;
    scale_factors<DT>(top, m0, m1);
#pragma unroll 2
    for (uint32_t i = tid; i < blocks * (kSlabUnit / 16); i += kSmallThreads) {
        const uint4 v = ld_shared(x + 16 * i);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t q[4];
        scale8<DT>(w, m0, m1, q, sum);
        st_shared(x + 16 * i, q[0], q[1], q[2], q[3]);
    }
    sum = block_sum32(sum);
    if (p.ctas > 1) {
        if (tid == 0) s_sum = sum;
        cluster_sync();
        sum = 0.0f;
        for (uint32_t q = 0; q < p.ctas; ++q) sum += __uint_as_float(ld_cluster_u32(cluster_addr(smem_u32(&s_sum), q)));
    }
    const float g0 = inverse_norm(sum, top, infinity_pattern<DT>());

    // Products: every thread's writes before it are seen by the tensor cores,
    // one thread issues, all wait.
    uint32_t parity = 0;
    const uint32_t steps_k = (p.side + 15) / 16;
    auto begin = [&]() {
        proxy_fence_shared();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    };
    auto finish = [&]() {
        bar_wait(bar, parity, quit);
        parity ^= 1;
        tc_fence_after();
    };
    constexpr uint32_t kIdesc = (1u << 4) | (static_cast<uint32_t>(kSide >> 4) << 24);   // fp32 = fp16 fp16, 128 rows
    constexpr uint32_t kIdesc128 = kIdesc | ((kSide >> 3) << 17), kMnA = 1u << 15, kMnB = 1u << 16;
    // this thread's part of a 128 x 128 result: 32 columns of a row
    const uint32_t row = (warp & 3) * 32 + lane, part = warp >> 2;
    const uint32_t my_tmem = tmem + part * 32 + ((warp & 3) << 21);

    // square `to` = f acc (+ f_lin `lin` + f_diag I), acc in the first 128 columns
    auto square_out = [&](uint32_t to, float f, bool poly, uint32_t lin, float f_lin, float f_diag) {
        uint32_t v[32];
        tmem_start32(my_tmem, v);
        tmem_wait(v);
        const bool diagonal = poly && part == (warp & 3);   // it crosses these rows in these columns
        const float d = row < p.side ? f_diag : 0.0f;
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) {
            const uint32_t piece = (part >> 1) * kBlockBytes + piece128(row, (part & 1) * 4 + j);
            float y[8];
#pragma unroll
            for (uint32_t e = 0; e < 8; ++e) y[e] = __uint_as_float(v[8 * j + e]) * f;
            if (poly) {
                const uint4 l = ld_shared(lin + piece);
                const uint32_t lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
                for (uint32_t e = 0; e < 4; ++e) {
                    float lo, hi;
                    widen2<kFp16>(lw[e], lo, hi);
                    y[2 * e] = __fmaf_rn(lo, f_lin, y[2 * e]);
                    y[2 * e + 1] = __fmaf_rn(hi, f_lin, y[2 * e + 1]);
                }
                if (diagonal) {   // added to every value, zero or not: a test of each turns into a branch a lane
#pragma unroll
                    for (uint32_t e = 0; e < 8; ++e) y[e] += lane == 8 * j + e ? d : 0.0f;
                }
            }
            st_shared(to + piece, narrow2<kFp16>(y[0], y[1]), narrow2<kFp16>(y[2], y[3]), narrow2<kFp16>(y[4], y[5]),
                      narrow2<kFp16>(y[6], y[7]));
        }
    };
    // the first square = f X X^T (or X^T X), summed over the cluster
    auto gram = [&](float f) {
        begin();
        if (warp == 0 && elect_one()) {
            // 16 of the longer side a product: 32 bytes of a wide block's rows, 16 rows of a tall one's blocks
            const uint64_t d0 = operand_desc(x, block_bytes);
            const uint32_t idesc = kIdesc128 | (tall ? kMnA | kMnB : 0u);
#pragma unroll 4
            for (uint32_t k = 0; k < blocks * 4; ++k) {
                const uint64_t d = d0 + (tall ? k * (2048 >> 4) : (k >> 2) * (kBlockBytes >> 4) + (k & 3) * 2);
                mma_f16(tmem, d, d, idesc, k > 0);
            }
            tc_commit(bar);
        }
        finish();
        if (p.ctas == 1) return;
        // the partial sums in fp32 where the other squares are, which are free here
        const uint32_t partial = sq0 + kSquareBytes;
        float v[32];
        tmem_load32(my_tmem, v);
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j)   // pieces of 4 columns, rotated by the row against bank conflicts
            st_shared(partial + row * 512 + (((part * 8 + j) ^ (row & 7)) << 4), __float_as_uint(v[4 * j]),
                      __float_as_uint(v[4 * j + 1]), __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3]));
        cluster_sync();
        // every CTA adds up some of the sums, in order of rank, and gives them to all; what is past the matrix's side
        // stays the zeros that it began with
        const uint32_t quads = (p.side + 3) / 4, sums = p.side * quads;
#pragma unroll 1
        for (uint32_t i = rank * kSmallThreads + tid; i < sums; i += p.ctas * kSmallThreads) {
            const uint32_t r = i / quads, c4 = i - r * quads;
            const uint32_t at = partial + r * 512 + ((c4 ^ (r & 7)) << 4);
            float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
            for (uint32_t q0 = 0; q0 < p.ctas; q0 += 4) {
                float4 y[4];
#pragma unroll
                for (uint32_t q = 0; q < 4; ++q)   // all on their way before the first is added
                    y[q] = q0 + q < p.ctas ? ld_cluster(cluster_addr(at, q0 + q)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (uint32_t q = 0; q < 4; ++q) {
                    s.x += y[q].x; s.y += y[q].y; s.z += y[q].z; s.w += y[q].w;
                }
            }
            const uint32_t lo = narrow2<kFp16>(s.x * f, s.y * f), hi = narrow2<kFp16>(s.z * f, s.w * f);
            const uint32_t to = sq0 + (c4 >> 4) * kBlockBytes + piece128(r, (c4 & 15) >> 1) + 8 * (c4 & 1);
#pragma unroll 1
            for (uint32_t q = 0; q < p.ctas; ++q) st_cluster(cluster_addr(to, q), lo, hi);
        }
        proxy_fence();
        cluster_sync();
    };
    // X = f B X (or X B) in place, or as bf16 for the caller
    auto update = [&](uint32_t m, float f, bool final) {
        begin();
        if (warp == 0 && elect_one()) {
            const uint64_t dm = operand_desc(m, 0), dx = operand_desc(x, block_bytes);
#pragma unroll 1
            for (uint32_t n0 = 0; n0 < blocks; n0 += tall ? 2 : 4) {   // 256 columns, or 128 rows, at a time
                const uint32_t idesc = tall ? kIdesc128 : kIdesc | kMnB | ((min(4u, blocks - n0) * 8) << 17);
#pragma unroll 2
                for (uint32_t k = 0; k < steps_k; ++k) {
                    const uint64_t square = dm + (k >> 2) * (kBlockBytes >> 4) + (k & 3) * 2;
                    if (tall)
                        mma_f16(tmem + n0 * 64, dx + n0 * (8192 >> 4) + (k >> 2) * (block_bytes >> 4) + (k & 3) * 2, square,
                                idesc, k > 0);
                    else
                        mma_f16(tmem + n0 * 64, square, dx + n0 * (kBlockBytes >> 4) + k * (2048 >> 4), idesc, k > 0);
                }
            }
            tc_commit(bar);
        }
        finish();
#pragma unroll 1
        for (uint32_t n = part; n < 2 * blocks; n += 4) {   // 32 columns of tensor memory each
            uint32_t v[32];
            tmem_start32(tmem + n * 32 + ((warp & 3) << 21), v);
            tmem_wait(v);
            const uint32_t to_row = tall ? (n >> 2) * 128 + row : row, to_col = (tall ? n & 3 : n) * 32;
            const uint32_t to = x + (to_col >> 6) * block_bytes;
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j) {
                uint32_t q[4];
#pragma unroll
                for (uint32_t e = 0; e < 4; ++e) {
                    const float lo = __uint_as_float(v[8 * j + 2 * e]) * f, hi = __uint_as_float(v[8 * j + 2 * e + 1]) * f;
                    q[e] = final ? narrow2<kBf16>(lo, hi) : narrow2<kFp16>(lo, hi);
                }
                st_shared(to + piece128(to_row, ((to_col & 63) >> 3) + j), q[0], q[1], q[2], q[3]);
            }
        }
    };

#pragma unroll 1
    for (int k = 0; k < p.steps;) {
        const bool raw = k == 0, pair = raw && p.steps >= 2;
        const float f_gram = raw ? kScaleA * g0 * g0 : kScaleA / (kScaleX * kScaleX);
        gram(f_gram);
        // The square products that follow: B = p(A) alone, or B, B A, A_1 = B (B A), B_1 = p(A_1), Q = B_1 B.  Each
        // digit of the three numbers is one of the squares: the result's, and the operands'.  Before them, without
        // a cluster, the Gram matrix's own rounding.
        const uint32_t products = pair ? 5 : 1;
#pragma unroll 1
        for (uint32_t i = p.ctas == 1 ? 0 : 1; i <= products; ++i) {
            const uint32_t digit = 4 * (i - 1);
            const uint32_t to = i == 0 ? 0u : (0x02021u >> digit) & 15u;
            const uint32_t a = sq0 + (i == 0 ? 0u : (0x20110u >> digit) & 15u) * kSquareBytes;
            const uint32_t c = sq0 + (i == 0 ? 0u : (0x10200u >> digit) & 15u) * kSquareBytes;
            const bool poly = i == 1 || i == 4;
            const float* co = s_coeffs + 3 * (k + (i == 4 ? 1 : 0));
            if (i > 0) {
                begin();
                if (warp == 0 && elect_one()) {
                    const uint64_t da = operand_desc(a, 0), dc = operand_desc(c, 0);
#pragma unroll 2
                    for (uint32_t s = 0; s < steps_k; ++s) {
                        const uint32_t at = (s >> 2) * (kBlockBytes >> 4) + (s & 3) * 2;
                        mma_f16(tmem, da + at, dc + at, kIdesc128, s > 0);
                    }
                    tc_commit(bar);
                }
                finish();
            }
            square_out(sq0 + to * kSquareBytes,
                       i == 0 ? f_gram : poly ? co[2] * (kScaleB / (kScaleA * kScaleA)) : 1.0f / kScaleB, poly, a,
                       co[1] * (kScaleB / kScaleA), co[0] * kScaleB);
        }
        k += pair ? 2 : 1;
        const bool final = k >= p.steps;
        update(sq0 + (pair ? 0u : kSquareBytes),
               (final ? p.scale : kScaleX) / (raw ? kScaleB : kScaleB * kScaleX) * (raw ? g0 : 1.0f), final);
    }
    __syncthreads();

    // to the caller's matrix
    {
        unsigned short* dst = static_cast<unsigned short*>(p.dst[b]) + (tall ? first * p.ld_dst : first);
        if ((reinterpret_cast<uintptr_t>(dst) & 15) == 0 && p.ld_dst % 8 == 0) {
#pragma unroll 1
            for (uint32_t i = tid; i < rows * eights; i += kSmallThreads) {
                const uint32_t r = i / eights, c = (i - r * eights) * 8;
                const uint4 v = ld_shared(place(r, c));
                unsigned short* out = dst + r * p.ld_dst + c;
                if (c + 8 <= cols) {
                    *reinterpret_cast<uint4*>(out) = v;
                } else {
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (uint32_t e = 0; e < 8; ++e)
                        if (c + e < cols) out[e] = static_cast<unsigned short>(w[e >> 1] >> (16 * (e & 1)));
                }
            }
        } else {   // aligned pieces of a row, of which the first and the last may be cut (73 us, by value 83)
            const uint32_t pieces = (cols + 14) / 8;
#pragma unroll 1
            for (uint32_t i = tid; i < rows * pieces; i += kSmallThreads) {
                const uint32_t r = i / pieces;
                unsigned short* row_out = dst + r * p.ld_dst;
                const uint32_t m = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row_out) >> 1) & 7u;
                const int c = static_cast<int>((i - r * pieces) * 8 - m);   // the piece's first column
                if (c >= static_cast<int>(cols)) continue;
                // the two eights that it lies in; the second only as far as the row goes
                const uint4 hi = ld_shared(place(r, min(static_cast<uint32_t>(c + 7), cols - 1) & ~7u));
                const uint4 lo = c < 0 ? hi : ld_shared(place(r, static_cast<uint32_t>(c) & ~7u));
                const uint32_t lw[4] = {lo.x, lo.y, lo.z, lo.w}, hw[4] = {hi.x, hi.y, hi.z, hi.w};
                uint32_t w[4];
                shift_halves(lw, hw, (8 - m) & 7, w);
                if (c >= 0 && c + 8 <= static_cast<int>(cols)) {
                    *reinterpret_cast<uint4*>(row_out + c) = make_uint4(w[0], w[1], w[2], w[3]);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (c + e >= 0 && c + e < static_cast<int>(cols))
                            row_out[c + e] = static_cast<unsigned short>(w[e >> 1] >> (16 * (e & 1)));
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    settle(quit);
    note_gave_up(quit, p.pending);
    if (p.ctas > 1) cluster_sync();   // nobody reads this CTA's shared memory any more
    if (warp == 0) {
        tc_fence_after();
        tmem_free(tmem, 512);
    }
}

// -------------------------------------------------------------------- host
// Blocks of the packing pass for one matrix: a unit a warp.
uint64_t pack_blocks(uint64_t rows, uint64_t cols) {
    const uint64_t units = (rows + kPackRows - 1) / kPackRows * ((cols + 255) / 256);
    return (units + kPackWarps - 1) / kPackWarps;
}

// The scratch of a call, as offsets from its start.
struct Scratch {
    uint64_t top, sum, ticket, g0, done, x[2], s[3], bytes;
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
    z.top = take(batch * kTopBlocks * sizeof(uint32_t));
    z.sum = take(batch * pack_blocks(rows, cols) * sizeof(float));
    z.ticket = take(batch * sizeof(uint32_t));
    z.g0 = take(batch * sizeof(float));
    z.done = take(batch * kMaxPhases * sizeof(uint32_t));
    for (uint64_t& x : z.x) x = take(batch * rows * up(cols, 8) * 2);
    for (uint64_t& s : z.s) s = take(batch * side * up(side, 8) * 2);
    z.bytes = at;
    return z;
}

// CTA pairs that can be resident at once on the current device.
cudaError_t pairs(int* out) {
    static std::mutex mu;
    static int known[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!known[dev]) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(kProductThreads);
        cfg.dynamicSmemBytes = kProductSmem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if ((e = cudaOccupancyMaxActiveClusters(&n, k_ortho_products, &cfg)) != cudaSuccess) return e;
        if (n < 1) return cudaErrorLaunchOutOfResources;
        known[dev] = n;
    }
    *out = known[dev];
    return cudaSuccess;
}

// Clusters of kMaxCtas CTAs of k_ortho_small that can be resident at once on the current device (none on one whose SMs
// do not come in groups that large).
template <int DT>
cudaError_t large_clusters(size_t smem, int* out) {
    static std::mutex mu;
    static int known[64] = {};   // and one
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!known[dev]) {
        if ((e = cudaFuncSetAttribute(k_ortho_small<DT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess)
            return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kMaxCtas);
        cfg.blockDim = dim3(kSmallThreads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = kMaxCtas;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if ((e = cudaOccupancyMaxActiveClusters(&n, k_ortho_small<DT>, &cfg)) != cudaSuccess) return e;
        known[dev] = n + 1;
    }
    *out = known[dev] - 1;
    return cudaSuccess;
}

constexpr float kDefaultCoeffs[3] = {3.4445f, -4.7750f, 2.0315f};

// Both calls; `pending` is the word of a step's state that learns of a wait that gave up, or NULL.
int orthogonalize(int dtype, int batch, uint64_t rows, uint64_t cols, const void* const* src, uint64_t ld_src,
                  void* const* dst, uint64_t ld_dst, int steps, const float* coeffs, float scale, void* workspace,
                  uint64_t workspace_bytes, int32_t* pending, void* stream) {
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
    for (int i = 0; i < batch; ++i) {
        if (!src[i] || !aligned(src[i], 2)) return refuse(ZERO_EINVAL, "src[i] is NULL or not 2-byte aligned");
        if (!dst[i] || !aligned(dst[i], 2)) return refuse(ZERO_EINVAL, "dst[i] is NULL or not 2-byte aligned");
    }
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

    cudaError_t e;
    constexpr size_t most_small = 1024 + 3 * kSquareBytes + kSlabBlocks * kSlabUnit;
    static_assert(most_small >= kAloneSmem, "the limit that is set covers every launch");
    uint32_t max_ctas = 0;   // of k_ortho_small for a matrix; none: too large for it
    if (side <= kSide && span <= kMaxCtas * kSlabBlocks * 64) {
        const bool fp16 = dtype == ZERO_FP16;
        if ((e = fp16 ? allow_smem<k_ortho_small<kFp16>>(most_small) : allow_smem<k_ortho_small<kBf16>>(most_small)) != cudaSuccess)
            return cuda_refuse(e, "zero_orthogonalize");
        max_ctas = span <= kPortableCtas * kSlabBlocks * 64 ? kPortableCtas : 0;
        if (span > kPortableCtas * 4 * 64) {
            int room = 0;
            if ((e = fp16 ? large_clusters<kFp16>(most_small, &room) : large_clusters<kBf16>(most_small, &room)) != cudaSuccess)
                return cuda_refuse(e, "zero_orthogonalize");
            if (max_ctas == 0 ? room > 0 : nb <= static_cast<uint32_t>(room)) max_ctas = kMaxCtas;
        }
    }
    if (max_ctas) {
        SmallArgs m = {};
        for (int i = 0; i < batch; ++i) {
            m.src[i] = src[i];
            m.dst[i] = dst[i];
        }
        m.ld_src = ld_src;
        m.ld_dst = ld_dst;
        m.side = static_cast<uint32_t>(side);
        m.span = static_cast<uint32_t>(span);
        const uint32_t blocks = (m.span + 63) / 64;
        // One CTA where it holds all: it sums nothing over a cluster (128 x 512 35 us, in two CTAs 39; 128 x 320 29, 36;
        // only a narrow side gains from more, 24 x 500 by 2 us).  Else 2 blocks of 64 a CTA on an empty GPU (2 x
        // 609 x 39 32 us, with 4 37; 23 x 1519 by 2 us), where clusters of that many find room side by side (16 x 64 x
        // 1000 took 61 so, with 4 32); then 4 as long as there are SMs, else as many as fit (16 x 64 x 1000 38 with 8).
        int sms = 0;
        if ((e = sm_count(&sms)) != cudaSuccess) return cuda_refuse(e, "zero_orthogonalize");
        const uint32_t halves = (blocks + 1) / 2 < max_ctas ? (blocks + 1) / 2 : max_ctas;
        m.ctas = blocks <= kSlabBlocks ? 1 : 2 * halves * nb <= static_cast<uint32_t>(sms) ? halves : (blocks + 3) / 4;
        if (m.ctas > max_ctas) m.ctas = max_ctas;
        while (m.ctas > 1 && m.ctas * nb > static_cast<uint32_t>(sms) && (m.ctas - 1) * kSlabBlocks >= blocks) --m.ctas;
        m.per = (blocks + m.ctas - 1) / m.ctas;
        if (tall) m.per += m.per & 1;            // 128 rows at a time
        m.ctas = (blocks + m.per - 1) / m.per;   // none without a block
        m.tall = tall;
        m.steps = steps;
        m.scale = scale;
        m.arrivals = take_matrix_hold() ? 2 : 1;
        m.pending = pending;
        for (int i = 0; i < 3 * steps; ++i) m.coeffs[i] = coeffs ? coeffs[i] : kDefaultCoeffs[i % 3];
        size_t smem = 1024 + 3 * kSquareBytes + static_cast<size_t>(m.per) * kSlabUnit;
        if (m.ctas > 1 && smem < kAloneSmem) smem = kAloneSmem;   // its blocks wait for one another: see tmem_alloc
        const dim3 grid(m.ctas * nb);
        e = dtype == ZERO_FP16 ? launch_pdl(k_ortho_small<kFp16>, grid, kSmallThreads, smem, m.ctas, s, m)
                               : launch_pdl(k_ortho_small<kBf16>, grid, kSmallThreads, smem, m.ctas, s, m);
        return e == cudaSuccess ? ZERO_OK : cuda_refuse(e, "zero_orthogonalize");
    }

    PackArgs q = {};
    ProductArgs p;   // its maps and phases are filled below
    std::memset(&p, 0, sizeof(p));
    p.dst_vec = ld_dst % 8 == 0;
    for (int i = 0; i < batch; ++i) {
        q.src[i] = src[i];
        p.dst[i] = dst[i];
        p.dst_vec &= aligned(dst[i], 16);
    }
    p.dst_ld = ld_dst;
    q.rows = rows;
    q.cols = cols;
    q.ld = ld_src;
    q.pitch = xp;
    q.segments = static_cast<uint32_t>((cols + 255) / 256);
    q.units = static_cast<uint32_t>((rows + kPackRows - 1) / kPackRows) * q.segments;
    q.top = reinterpret_cast<uint32_t*>(ws + z.top);
    q.sum = reinterpret_cast<float*>(ws + z.sum);
    q.ticket = reinterpret_cast<uint32_t*>(ws + z.ticket);
    q.g0 = reinterpret_cast<float*>(ws + z.g0);
    q.done = reinterpret_cast<uint32_t*>(ws + z.done);
    q.x0 = reinterpret_cast<__half*>(ws + z.x[0]);
    q.sums = static_cast<uint32_t>(pack_blocks(rows, cols));
    q.tops = q.sums < kTopBlocks ? q.sums : kTopBlocks;
    if ((e = launch_pdl(k_ortho_top, dim3(q.tops, nb), kThreads, 0, 1, s, q)) != cudaSuccess) return cuda_refuse(e, "scale");
    e = dtype == ZERO_FP16 ? launch_pdl(k_ortho_pack<kFp16>, dim3(q.sums, nb), kThreads, 0, 1, s, q)
                           : launch_pdl(k_ortho_pack<kBf16>, dim3(q.sums, nb), kThreads, 0, 1, s, q);
    if (e != cudaSuccess) return cuda_refuse(e, "pack");
    const uint64_t xs = rows * xp, ss = side * sp;
    for (int i = 0; i < 2; ++i) {
        const void* base = ws + z.x[i];
        if ((e = make_map(&p.maps[kXRows0 + i], 2, base, cols, rows, nb, xp, xs, kBlockK, kHalf)) != cudaSuccess ||
            (e = make_map(&p.maps[kXCols0 + i], 2, base, cols, rows, nb, xp, xs, 64, kBlockK)) != cudaSuccess ||
            (e = make_map(&p.maps[kXOut0 + i], 2, base, cols, rows, nb, xp, xs, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B)) !=
                cudaSuccess)
            return cuda_refuse(e, "tensor map");
    }
    for (int i = 0; i < 3; ++i) {
        const void* base = ws + z.s[i];
        if ((e = make_map(&p.maps[kSquare0 + i], 2, base, side, side, nb, sp, ss, kBlockK, kHalf)) != cudaSuccess ||
            (e = make_map(&p.maps[kSquareOut0 + i], 2, base, side, side, nb, sp, ss, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B)) !=
                cudaSuccess)
            return cuda_refuse(e, "tensor map");
    }
    p.g0 = q.g0;
    p.done = q.done;
    p.hold = take_matrix_hold();
    p.pending = pending;
    p.batch = nb;
    uint32_t most = 0;   // tiles of the largest phase

    auto square = [&](int to, int a, int b, uint64_t depth) -> Phase& {   // a symmetric product into square matrix `to`
        Phase& f = p.phases[p.n_phases++];
        const uint32_t t = static_cast<uint32_t>((side + kTile - 1) / kTile);
        f.a = a;
        f.b = b;
        f.out = kSquareOut0 + to;
        f.symmetric = 1;
        f.epi = kScale;
        f.rows = f.cols = static_cast<uint32_t>(side);
        f.depth = static_cast<uint32_t>(depth);
        f.tiles_n = t;
        f.tiles = t * (t + 1) / 2;
        most = f.tiles > most ? f.tiles : most;
        return f;
    };
    // A = X X^T or X^T X of X buffer `x` into `to`; `raw`: that buffer still holds X0
    auto gram = [&](int to, int x, bool raw) {
        const int map = (tall ? kXCols0 : kXRows0) + x;
        Phase& f = square(to, map, map, span);
        f.a_mn = f.b_mn = tall;
        f.f_acc = raw ? kScaleA : kScaleA / (kScaleX * kScaleX);
        f.g_power = raw ? 2 : 0;
    };
    // to = a I + b A + c A^2
    auto poly = [&](int to, int a, const float* c) {
        Phase& f = square(to, kSquare0 + a, kSquare0 + a, side);
        f.epi = kPoly;
        f.lin = kSquareOut0 + a;
        f.f_diag = c[0] * kScaleB;
        f.f_lin = c[1] * (kScaleB / kScaleA);
        f.f_acc = c[2] * (kScaleB / (kScaleA * kScaleA));
    };
    // to = B M, two commuting symmetric matrices, B of scale kScaleB
    auto commuting = [&](int to, int b, int m) {
        square(to, kSquare0 + b, kSquare0 + m, side).f_acc = 1.0f / kScaleB;
    };
    // the other X buffer (or dst) = B X, or X B of a tall matrix
    auto apply = [&](int x, int b, bool raw, bool to_dst) {
        Phase& f = p.phases[p.n_phases++];
        f.a = tall ? kXRows0 + x : kSquare0 + b;
        f.b = tall ? kSquare0 + b : kXCols0 + x;
        f.b_mn = !tall;
        f.out = kXOut0 + (x ^ 1);
        f.epi = to_dst ? kFinal : kScale;
        f.rows = static_cast<uint32_t>(rows);
        f.cols = static_cast<uint32_t>(cols);
        f.depth = static_cast<uint32_t>(side);
        f.tiles_n = (f.cols + kTile - 1) / kTile;
        f.tiles = f.tiles_n * ((f.rows + kTile - 1) / kTile);
        most = f.tiles > most ? f.tiles : most;
        f.g_power = raw ? 1 : 0;
        f.f_acc = (to_dst ? scale : kScaleX) / (raw ? kScaleB : kScaleB * kScaleX);
    };

    int x = 0;
    for (int k = 0; k < steps;) {
        const float* c = coeffs ? coeffs + 3 * k : kDefaultCoeffs;
        const bool raw = k == 0, pair = raw && steps >= 2;
        gram(0, x, raw);
        poly(1, 0, c);
        int b = 1;
        if (pair) {
            commuting(2, 1, 0);                             // B A
            commuting(0, 1, 2);                             // A_1 = B (B A)
            poly(2, 0, coeffs ? coeffs + 3 : kDefaultCoeffs);
            commuting(0, 2, 1);                             // Q = B_1 B
            b = 0;
        }
        k += pair ? 2 : 1;
        apply(x, b, raw, k >= steps);
        x ^= 1;
    }

    int resident = 0;
    if ((e = allow_smem<k_ortho_products>(kProductSmem)) != cudaSuccess || (e = pairs(&resident)) != cudaSuccess)
        return cuda_refuse(e, "zero_orthogonalize");
    const uint64_t tiles = static_cast<uint64_t>(most) * nb;
    // Every pair, also where no phase has a tile for each: consecutive phases then run on different pairs, and a tile
    // finds its pair at rest (9 x 303 x 374: 133 us against 141 with a pair a tile, 3 x 477 x 650: 149 against 159).
    // A single tile stays where it is (235 x 142: 101.5 against 104.9).
    const unsigned grid = 2u * static_cast<unsigned>(tiles > 1 ? resident : 1);
    e = launch_together(k_ortho_products, dim3(grid), kProductThreads, kProductSmem, 2, s, p);
    if (e != cudaSuccess) return cuda_refuse(e, "products");
    return ZERO_OK;
}

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
    return orthogonalize(dtype, batch, rows, cols, src, ld_src, dst, ld_dst, steps, coeffs, scale, workspace,
                         workspace_bytes, nullptr, stream);
}

int zero_muon_orthogonalize(int dtype, int batch, uint64_t rows, uint64_t cols, const void* const* src, uint64_t ld_src,
                            void* const* dst, uint64_t ld_dst, int steps, const float* coeffs, float scale,
                            void* workspace, uint64_t workspace_bytes, zero_muon_state_t* state, void* stream) {
    if (!state || !aligned(state, 8)) return refuse(ZERO_EINVAL, "state is NULL or not 8-byte aligned");
    return orthogonalize(dtype, batch, rows, cols, src, ld_src, dst, ld_dst, steps, coeffs, scale, workspace,
                         workspace_bytes, &state->pending, stream);
}

}  // extern "C"
