// The streams around an orthogonalised update (Muon): the ranks' gradients
// into the momentum, and the finished update into the master and every
// rank's 16-bit replica.
//
//   momentum  g = (sum over ranks, in rank order, of f32(g_r)) / (N * scale)
//             m' = mu m + g;   u = g + mu m' (Nesterov) or m', rounded to bf16
//   apply     w = (1 - lr wd) w - lr o;   every replica = round16(w)
//
// Both are bound by HBM: 2N + 10 and 10 + 2N bytes an element, every byte
// touched once.  Measured: the 84,934,656 elements of GPT-2 small's hidden
// matrices on 8 ranks take the momentum 308 us (7.2 TB/s, mostly reads), a
// Llama-7B layer's 202,375,168 on 8 ranks take apply 780 us (6.7 TB/s); a
// plain copy moves 6.8 TB/s.  A thread moves 8 elements (256-bit fp32 accesses where the
// buffers allow), with the loads of up to 8 ranks in flight together, as
// the AdamW step's kernels do.  The grid is not persistent: a block handles
// kMuonVecs vectors a thread and leaves, so that the hardware hands out the
// work and no SM idles while others still stream.
//
// Whether a gradient overflowed is known only when all were read, but the
// momentum is written on the way.  It therefore has two slots: the new
// momentum goes to the slot that is not live, and zero_muon_apply makes that
// slot the live one or, after an overflow, leaves everything as it was.  The
// same holds where the orthogonalisation between them could not finish.

#include <cmath>
#include <cstdint>
#include <string>

#include <nvtx3/nvToolsExt.h>

#include "zero_gb300.h"
#include "zero_host.h"
#include "zero_device.cuh"

namespace zg {
namespace {

constexpr int kMuonVecs = 2;

struct MuonArgs {
    const void* grads[kMaxRanks];
    void* params[kMaxRanks];
    int n_ranks;
    uint64_t count;
    uint64_t slot_stride;   // floats between the momentum's slots
    float* momentum;
    float* master;
    void* update;           // written by momentum (u), read by apply (o); bf16
    float mu, lr, dfac;     // dfac = 1 - lr wd, rounded once from double
    int nesterov;
    zero_muon_state_t* state;
};

struct MuonPro {
    float den, inv;
    int use_div, slot, skip;   // skip: the state's `pending`
};

// The unscale factor N * scale and the live slot, read once per block.
__device__ __forceinline__ void muon_prologue(const MuonArgs& a, MuonPro& pro) {
    if (threadIdx.x == 0) {
        const float den = __fmul_rn(static_cast<float>(a.n_ranks), a.state->loss_scale);
        const uint32_t bits = __float_as_uint(den), ex = (bits >> 23) & 0xFFu;
        // a power of two with a normal reciprocal: multiplying by it is the division
        const bool pow2 = (bits & 0x7FFFFFu) == 0u && ex >= 1u && ex <= 253u;
        pro.den = den;
        pro.use_div = pow2 ? 0 : 1;
        pro.inv = pow2 ? __fdiv_rn(1.0f, den) : 0.0f;
        pro.slot = a.state->slot & 1;
        pro.skip = a.state->pending;
    }
    __syncthreads();
}

template <int DT, class IO>
__device__ __forceinline__ bool momentum_at(const MuonArgs& a, const MuonPro& pro, uint64_t i) {
    constexpr int W = IO::W;
    const float* src = a.momentum + static_cast<uint64_t>(pro.slot) * a.slot_stride;
    float* dst = a.momentum + static_cast<uint64_t>(pro.slot ^ 1) * a.slot_stride;
    float m[W], s[W];
    IO::ldf(src, i, m);
#pragma unroll
    for (int k = 0; k < W; ++k) s[k] = 0.0f;
    const int n = a.n_ranks;
    int r = 0;
    for (; r + 8 <= n; r += 8) {
        uint32_t raw[8][W];
#pragma unroll
        for (int q = 0; q < 8; ++q) IO::ld16(a.grads[r + q], i, raw[q]);
#pragma unroll
        for (int q = 0; q < 8; ++q)
#pragma unroll
            for (int k = 0; k < W; ++k) s[k] = __fadd_rn(s[k], widen<DT>(raw[q][k]));
    }
    for (; r < n; ++r) {
        uint32_t raw[W];
        IO::ld16(a.grads[r], i, raw);
#pragma unroll
        for (int k = 0; k < W; ++k) s[k] = __fadd_rn(s[k], widen<DT>(raw[k]));
    }
    bool bad = false;
    uint32_t u[W];
#pragma unroll
    for (int k = 0; k < W; ++k) {
        const float g = pro.use_div ? __fdiv_rn(s[k], pro.den) : __fmul_rn(s[k], pro.inv);
        bad |= nonfinite(g);
        m[k] = __fadd_rn(__fmul_rn(a.mu, m[k]), g);
        u[k] = narrow<kBf16>(a.nesterov ? __fadd_rn(g, __fmul_rn(a.mu, m[k])) : m[k]);
    }
    IO::stf(dst, i, m);
    IO::st16(a.update, i, u);
    return bad;
}

template <int DT, class IO>
__global__ void __launch_bounds__(kThreads) k_muon_momentum(const __grid_constant__ MuonArgs a) {
    pdl_enter();
    __shared__ MuonPro pro;
    muon_prologue(a, pro);
    const uint64_t nvec = a.count / IO::W, rest = a.count - nvec * IO::W;
    const uint64_t v0 = static_cast<uint64_t>(blockIdx.x) * kMuonVecs * kThreads + threadIdx.x;
    bool bad = false;
#pragma unroll
    for (int k = 0; k < kMuonVecs; ++k) {
        const uint64_t v = v0 + static_cast<uint64_t>(k) * kThreads;
        if (v < nvec) bad |= momentum_at<DT, IO>(a, pro, v * IO::W);
    }
    // the last, partial vector: one element a thread of the last block
    if (IO::W > 1 && blockIdx.x == gridDim.x - 1 && threadIdx.x < rest)
        bad |= momentum_at<DT, Io1>(a, pro, nvec * IO::W + threadIdx.x);
    if (bad) atomicOr(reinterpret_cast<int*>(&a.state->pending), ZERO_MUON_NONFINITE);
}

template <int DT, class IO>
__device__ __forceinline__ void apply_at(const MuonArgs& a, uint64_t i) {
    constexpr int W = IO::W;
    float w[W];
    uint32_t o[W], q[W];
    IO::ldf(a.master, i, w);
    IO::ld16(a.update, i, o);
#pragma unroll
    for (int k = 0; k < W; ++k) {
        w[k] = __fsub_rn(__fmul_rn(w[k], a.dfac), __fmul_rn(a.lr, widen<kBf16>(o[k])));
        q[k] = narrow<DT>(w[k]);
    }
    IO::stf(a.master, i, w);
    for (int r = 0; r < a.n_ranks; ++r) IO::st16(a.params[r], i, q);
}

// The last block to finish turns the step's outcome into the state: applied
// (the momentum's new slot becomes live) or skipped (the loss scale halves if
// a gradient was the reason).
template <int DT, class IO>
__global__ void __launch_bounds__(kThreads) k_muon_apply(const __grid_constant__ MuonArgs a) {
    pdl_enter();
    __shared__ MuonPro pro;
    muon_prologue(a, pro);
    if (!pro.skip) {
        const uint64_t nvec = a.count / IO::W, rest = a.count - nvec * IO::W;
        const uint64_t v0 = static_cast<uint64_t>(blockIdx.x) * kMuonVecs * kThreads + threadIdx.x;
#pragma unroll
        for (int k = 0; k < kMuonVecs; ++k) {
            const uint64_t v = v0 + static_cast<uint64_t>(k) * kThreads;
            if (v < nvec) apply_at<DT, IO>(a, v * IO::W);
        }
        if (IO::W > 1 && blockIdx.x == gridDim.x - 1 && threadIdx.x < rest)
            apply_at<DT, Io1>(a, nvec * IO::W + threadIdx.x);
    }
    if (threadIdx.x == 0) {
        // every block has read `pending` and `slot` before its ticket
        __threadfence();
        if (atomicAdd(&a.state->ticket, 1u) == gridDim.x - 1) {
            zero_muon_state_t* st = a.state;
            st->ticket = 0u;
            st->overflow = pro.skip != 0;
            st->applied = pro.skip == 0;
            st->aborted = (pro.skip & ZERO_MUON_GAVE_UP) != 0;
            if (pro.skip) {
                if (pro.skip & ZERO_MUON_NONFINITE) st->loss_scale = fmaxf(__fmul_rn(st->loss_scale, 0.5f), 1.0f);
                st->steps_skipped += 1;
            } else {
                st->slot = pro.slot ^ 1;
                st->steps_applied += 1;
            }
            st->pending = 0;
        }
    }
}

__global__ void k_muon_set_state(zero_muon_state_t* st, float loss_scale, int64_t t, int32_t slot) {
    pdl_enter();
    zero_muon_state_t z = {};
    z.loss_scale = loss_scale;
    z.steps_applied = t;
    z.slot = slot;
    *st = z;
}

template <int DT>
cudaError_t launch_momentum(const MuonArgs& a, bool v32, unsigned blocks, cudaStream_t s) {
    return v32 ? launch_pdl(k_muon_momentum<DT, Io8s32>, dim3(blocks), kThreads, 0, 1, s, a)
               : launch_pdl(k_muon_momentum<DT, Io8s16>, dim3(blocks), kThreads, 0, 1, s, a);
}
template <int DT>
cudaError_t launch_apply(const MuonArgs& a, bool v32, unsigned blocks, cudaStream_t s) {
    return v32 ? launch_pdl(k_muon_apply<DT, Io8s32>, dim3(blocks), kThreads, 0, 1, s, a)
               : launch_pdl(k_muon_apply<DT, Io8s16>, dim3(blocks), kThreads, 0, 1, s, a);
}

// What both calls check; fills what both kernels take.
int muon_args(MuonArgs& a, int dtype, int n_ranks, uint64_t count, const zero_muon_hyper_t* hyper,
              zero_muon_state_t* state) {
    if (dtype != ZERO_FP16 && dtype != ZERO_BF16) return refuse(ZERO_EINVAL, "dtype must be fp16 or bf16");
    if (n_ranks < 1 || n_ranks > ZERO_MAX_RANKS) return refuse(ZERO_EINVAL, "n_ranks must be in 1..64");
    if (count > (1ull << 40)) return refuse(ZERO_EINVAL, "count too large");
    if (!hyper) return refuse(ZERO_EINVAL, "hyper is NULL");
    const float hv[] = {hyper->lr, hyper->momentum, hyper->weight_decay};
    for (float x : hv)
        if (!std::isfinite(x)) return refuse(ZERO_EINVAL, "hyper-parameters must be finite");
    if (!(hyper->momentum >= 0.0f && hyper->momentum < 1.0f)) return refuse(ZERO_EINVAL, "momentum must lie in [0, 1)");
    if (!state || !aligned(state, 8)) return refuse(ZERO_EINVAL, "state is NULL or not 8-byte aligned");
    a.n_ranks = n_ranks;
    a.count = count;
    a.slot_stride = (count + 7) / 8 * 8;
    a.mu = hyper->momentum;
    a.lr = hyper->lr;
    a.dfac = static_cast<float>(1.0 - static_cast<double>(hyper->lr) * static_cast<double>(hyper->weight_decay));
    a.nesterov = hyper->nesterov != 0;
    a.state = state;
    return ZERO_OK;
}

unsigned muon_blocks(uint64_t count) {
    const uint64_t per = static_cast<uint64_t>(kThreads) * kMuonVecs * 8;
    const uint64_t b = (count + per - 1) / per;
    return static_cast<unsigned>(b < 1 ? 1 : b);
}

}  // namespace
}  // namespace zg

using namespace zg;

extern "C" {

int zero_muon_set_state(zero_muon_state_t* state, float loss_scale, int64_t steps_applied, int32_t slot, void* stream) {
    if (!state || !aligned(state, 8)) return refuse(ZERO_EINVAL, "state is NULL or not 8-byte aligned");
    if (!(loss_scale > 0.0f) || !std::isfinite(loss_scale))
        return refuse(ZERO_EINVAL, "loss_scale must be finite and > 0");
    if (steps_applied < 0) return refuse(ZERO_EINVAL, "steps_applied must be >= 0");
    if (slot != 0 && slot != 1) return refuse(ZERO_EINVAL, "slot must be 0 or 1");
    const cudaError_t e = launch_pdl(k_muon_set_state, dim3(1), 1, 0, 1, static_cast<cudaStream_t>(stream), state,
                                     loss_scale, steps_applied, slot);
    return e == cudaSuccess ? ZERO_OK : cuda_refuse(e, "zero_muon_set_state");
}

int zero_muon_get_state(const zero_muon_state_t* state, void* stream, zero_muon_state_t* out) {
    if (!state || !aligned(state, 8)) return refuse(ZERO_EINVAL, "state is NULL or not 8-byte aligned");
    if (!out) return refuse(ZERO_EINVAL, "out is NULL");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemcpyAsync(out, state, sizeof(*out), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    return e == cudaSuccess ? ZERO_OK : cuda_refuse(e, "zero_muon_get_state");
}

int zero_muon_momentum(int dtype, int n_ranks, uint64_t count, const void* const* grads, float* momentum,
                       void* update, const zero_muon_hyper_t* hyper, zero_muon_state_t* state, void* stream) {
    nvtxRangePushA("zero_muon_momentum");
    struct Pop { ~Pop() { nvtxRangePop(); } } pop;
    MuonArgs a = {};
    if (const int rc = muon_args(a, dtype, n_ranks, count, hyper, state)) return rc;
    if (count == 0) return ZERO_OK;
    if (!grads) return refuse(ZERO_EINVAL, "grads is NULL");
    for (int r = 0; r < n_ranks; ++r) {
        if (!grads[r] || !aligned(grads[r], 16)) return refuse(ZERO_EINVAL, "grads[r] is NULL or not 16-byte aligned");
        a.grads[r] = grads[r];
    }
    if (!momentum || !aligned(momentum, 16)) return refuse(ZERO_EINVAL, "momentum is NULL or not 16-byte aligned");
    if (!update || !aligned(update, 16)) return refuse(ZERO_EINVAL, "update is NULL or not 16-byte aligned");
    a.momentum = momentum;
    a.update = update;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool v32 = aligned(momentum, 32);
    const cudaError_t e = dtype == ZERO_FP16 ? launch_momentum<kFp16>(a, v32, muon_blocks(count), s)
                                             : launch_momentum<kBf16>(a, v32, muon_blocks(count), s);
    return e == cudaSuccess ? ZERO_OK : cuda_refuse(e, "zero_muon_momentum");
}

int zero_muon_apply(int dtype, int n_ranks, uint64_t count, const void* ortho, float* master, void* const* params,
                    const zero_muon_hyper_t* hyper, zero_muon_state_t* state, void* stream) {
    nvtxRangePushA("zero_muon_apply");
    struct Pop { ~Pop() { nvtxRangePop(); } } pop;
    MuonArgs a = {};
    if (const int rc = muon_args(a, dtype, n_ranks, count, hyper, state)) return rc;
    if (count > 0) {
        if (!params) return refuse(ZERO_EINVAL, "params is NULL");
        for (int r = 0; r < n_ranks; ++r) {
            if (!params[r] || !aligned(params[r], 16))
                return refuse(ZERO_EINVAL, "params[r] is NULL or not 16-byte aligned");
            a.params[r] = params[r];
        }
        if (!ortho || !aligned(ortho, 16)) return refuse(ZERO_EINVAL, "ortho is NULL or not 16-byte aligned");
        if (!master || !aligned(master, 16)) return refuse(ZERO_EINVAL, "master is NULL or not 16-byte aligned");
        a.update = const_cast<void*>(ortho);
        a.master = master;
    }
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool v32 = aligned(master, 32);
    const cudaError_t e = dtype == ZERO_FP16 ? launch_apply<kFp16>(a, v32, muon_blocks(count), s)
                                             : launch_apply<kBf16>(a, v32, muon_blocks(count), s);
    return e == cudaSuccess ? ZERO_OK : cuda_refuse(e, "zero_muon_apply");
}

}  // extern "C"
