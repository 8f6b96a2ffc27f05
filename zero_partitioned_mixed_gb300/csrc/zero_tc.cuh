// Tensor-core plumbing shared by the matrix kernels (zero_ortho.cu,
// zero_mx4.cu): tensor maps on the host; mbarriers with bounded waits, bulk
// tensor copies, and the tcgen05 instructions on the device.  Each
// translation unit gets its own copy (anonymous namespace).
//
// Operand tiles live in shared memory in the 128-byte swizzle, which both
// the bulk tensor copy and the matrix instructions apply by themselves:
//   * "K-major": a row of the tile is 128 bytes along the contraction, rows
//     follow each other, groups of 8 rows every 1024 bytes;
//   * "MN-major": a row is 64 16-bit values along the tile's own M or N, one
//     row per step of the contraction, groups of 8 steps every 1024 bytes,
//     the next 64 values of M or N a whole block further on.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "zero_host.h"
#include "zero_device.cuh"

namespace zg {
namespace {

// ------------------------------------------------------------ tensor maps
// cuTensorMapEncodeTiled, found through the runtime so that the library does
// not link against the driver.
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

// A [batch][rows][cols] array of `elem`-byte values (1 or 2) with `pitch` values between rows, read in boxes of box_cols x box_rows in
// the 128-byte swizzle (or another); what lies outside the array reads as zero.
inline cudaError_t make_map(CUtensorMap* map, int elem, const void* base, uint64_t cols, uint64_t rows, uint64_t batch,
                            uint64_t pitch, uint64_t matrix_stride, uint32_t box_cols, uint32_t box_rows,
                            CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B, uint32_t box_batch = 1) {
    const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {cols, rows, batch};
    const cuuint64_t strides[2] = {pitch * static_cast<uint64_t>(elem), matrix_stride * static_cast<uint64_t>(elem)};
    const cuuint32_t box[3] = {box_cols, box_rows, box_batch};
    const cuuint32_t step[3] = {1, 1, 1};
    const CUresult r = encode(map, elem == 2 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3,
                              const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// ---------------------------------------------------------------- barriers
// Waits for an mbarrier or a counter end by themselves after this time.  What
// has no limit: allocating tensor memory (see tmem_alloc), a cluster's barrier
// (its blocks run together, and between two barriers each has only waits of
// the first kind), and the waits for a block's own copies and loads, which
// the hardware completes.
constexpr uint64_t kGiveUpNs = 2000000000ull;

// What the first thread whose bounded wait gave up was waiting for (WaitFor);
// read and cleared by the host's status call.
__device__ int32_t g_gave_up;

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ uint64_t now_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_init_fence() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Whether the phase of parity `parity` is complete; may suspend the thread
// for up to kTryNs until it is.
constexpr uint32_t kTryNs = 20000;
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(kTryNs)
        : "memory");
    return ok != 0;
}
// One lane of a converged warp.  The compiler knows that a region under it has
// one thread, and keeps the operands of the copies and products issued there
// in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
// A place in a ring of N stages: its index, and the parity of its barriers'
// phase in this round.
template <uint32_t N>
struct Ring {
    uint32_t s = 0, parity = 0;
    __device__ __forceinline__ void next() {
        if (++s == N) {
            s = 0;
            parity ^= 1;
        }
    }
};
// What a thread was waiting for when it gave up (g_gave_up).
enum WaitFor : int32_t { kForSpace = 1, kForData = 2, kForProducts = 3, kForInputs = 4 };

__device__ __noinline__ void give_up(volatile int* quit, int32_t what) {
    *quit = 1;
    atomicCAS(&g_gave_up, 0, what);   // the first one is the one to look at
}
// Waits for the phase of parity `parity`; false when the wait gave up or
// another role of the block had (`*quit`).
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int* quit, int32_t what = kForProducts) {
    if (bar_test(bar, parity)) return true;
    const uint64_t t0 = now_ns();
    for (uint32_t i = 1;; ++i) {
        if (bar_test(bar, parity)) return true;
        if ((i & 15u) == 0u) {
            if (*quit) return false;
            if (now_ns() - t0 > kGiveUpNs) {
                give_up(quit, what);
                return false;
            }
        }
    }
}
// The same without regard to `quit`, until kGiveUpNs after t0: for the copies
// and products that a block still has in flight when it gives up.
__device__ __forceinline__ void bar_drain(uint32_t bar, uint32_t parity, uint64_t t0) {
    while (!bar_test(bar, parity) && now_ns() - t0 < kGiveUpNs) {}
}
// In every thread, after a barrier of the block behind which nobody waits any
// more: when a wait gave up, copies and products may still be in flight.  They
// land within microseconds and are left a millisecond, before the block frees
// its tensor memory or leaves.
__device__ __forceinline__ void settle(volatile int* quit) {
    if (!*quit) return;
    const uint64_t t0 = now_ns();
    while (now_ns() - t0 < 1000000ull) {}
    __syncwarp();
}

// ------------------------------------------------------------------ copies
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
// The same in a pair of CTAs: `dst` is this CTA's, `bar` (an address in the
// cluster's window) the leader's.
__device__ __forceinline__ void copy_box_pair(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void store_box(const CUtensorMap* map, int x, int y, int z, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
                 ::"l"(map), "r"(x), "r"(y), "r"(z), "r"(src)
                 : "memory");
}
__device__ __forceinline__ void store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// At most N of this thread's store groups still read shared memory / are unfinished.
template <int N>
__device__ __forceinline__ void store_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ void store_wait() {
    asm volatile("cp.async.bulk.wait_group %0;" ::"n"(N) : "memory");
}
// Ordinary accesses before it and bulk copies after it (or the reverse) are ordered.
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async;" ::: "memory"); }

__device__ __forceinline__ void proxy_fence_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }
__device__ __forceinline__ void proxy_fence_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// A shared-memory address of this CTA as it is in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 ld_cluster(uint32_t addr) {
    float4 x;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                 : "r"(addr)
                 : "memory");
    return x;
}
__device__ __forceinline__ void bar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Waits until the counter reaches `target` (a count of finished pieces of
// work of other blocks, released by count_done).
__device__ __forceinline__ bool count_wait(const uint32_t* counter, uint32_t target, volatile int* quit) {
    const uint64_t t0 = now_ns();
    for (uint32_t i = 1;; ++i) {
        uint32_t v;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(counter) : "memory");
        if (v >= target) return true;
        if ((i & 63u) == 0u) {
            if (*quit) return false;
            if (now_ns() - t0 > kGiveUpNs) {
                give_up(quit, kForInputs);
                return false;
            }
        }
    }
}
__device__ __forceinline__ void count_done(uint32_t* counter) {
    asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(counter) : "memory");
}
// ----------------------------------------------------------------- tcgen05
// A block allocates tensor memory before its pdl_enter(), with a block-wide
// barrier in between: the next kernel's blocks come only after every block of
// this one has passed pdl_enter(), so they cannot hold tensor memory that a
// block of this kernel still waits for while they themselves wait for it.
//
// That orders the kernels of one stream.  Between streams: an allocation has
// no time limit, nor has a cluster's barrier, so a block must not keep its
// tensor memory while it waits for another block, unless nothing that also
// allocates can be on its SM.  With two clusters of different kernels on the
// same two SMs, each could hold one and wait for the other, for ever.
// k_mx4_narrow frees before it waits for its cluster; the clusters of
// zero_ortho.cu ask for kAloneSmem of shared memory or more, which leaves no
// room on an SM for a block with kLeastTmemSmem, the least that a kernel here
// with tensor memory asks for.
constexpr size_t kSmemPerSm = 228 * 1024;   // each block takes 1 KiB more than it asks for
constexpr size_t kLeastTmemSmem = 60 * 1024, kAloneSmem = 168 * 1024;
static_assert(kAloneSmem + kLeastTmemSmem + 2 * 1024 > kSmemPerSm, "a block beside one of kAloneSmem");
__device__ __forceinline__ void tmem_alloc(uint32_t smem_slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_slot), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// The barrier gets one arrival once every product issued so far has finished.
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// D (fp32, tensor memory) = A B + (accumulate ? D : 0), 16-bit operands.
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
}
// The same instructions for a pair of CTAs: one product of 256 rows, each CTA
// holding 128 of A's rows, half of B's columns and 128 rows of D.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t smem_slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_slot), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free_pair(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
// One arrival at this barrier of both CTAs.
__device__ __forceinline__ void tc_commit_pair(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        ::"r"(bar), "h"(static_cast<uint16_t>(3))
        : "memory");
}
__device__ __forceinline__ void mma_f16_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
}
// 32 lanes x 32 columns of fp32: thread t gets lane (its warp's quarter) + t.
__device__ __forceinline__ void tmem_start32(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
// The registers are filled only after the wait, which therefore names them:
// nothing that reads them may move before it.
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28])
                 :
                 : "memory");
    asm volatile("" : "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}
__device__ __forceinline__ void tmem_load32(uint32_t addr, float (&v)[32]) {
    uint32_t r[32];
    tmem_start32(addr, r);
    tmem_wait(r);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// The same of 16 columns.
__device__ __forceinline__ void tmem_load16(uint32_t addr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;"   // names the registers: see tmem_wait
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// Shared-memory operand descriptor in the 128-byte swizzle.  `lead` is the
// distance in bytes between 64-value blocks of an MN-major tile (unused for
// K-major); groups of 8 rows are 1024 bytes apart in both.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t lead) {
    uint64_t d = static_cast<uint64_t>((addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>((lead >> 4) & 0x3FFFu) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;   // descriptor version of sm_100
    d |= static_cast<uint64_t>(2) << 61;   // 128-byte swizzle
    return d;
}

// Byte offset of 16-byte piece j of row r in a buffer of 128-byte or 64-byte
// rows, as the bulk copy's swizzle of that width places it.
__device__ __forceinline__ uint32_t piece128(uint32_t r, uint32_t j) { return r * 128 + ((j ^ (r & 7)) << 4); }
__device__ __forceinline__ uint32_t piece64(uint32_t r, uint32_t j) { return r * 64 + ((j ^ ((r >> 1) & 3)) << 4); }
__device__ __forceinline__ void st_shared(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void st_shared(uint32_t addr, uint32_t x) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}
__device__ __forceinline__ uint4 ld_shared(uint32_t addr) {
    uint4 x;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                 : "r"(addr)
                 : "memory");
    return x;
}
__device__ __forceinline__ uint16_t ld_shared16(uint32_t addr) {
    uint16_t x;
    asm volatile("ld.shared.b16 %0, [%1];" : "=h"(x) : "r"(addr) : "memory");
    return x;
}

// 32 rows x 32 columns of 16-bit values in a warp's buffer (piece64) into rows
// row0... and columns col0... of a row-major rows x cols matrix: 16 bytes a
// lane where every row starts on 16 bytes (`vec`), value by value elsewhere.
__device__ __forceinline__ void write_rows(unsigned short* dst, uint64_t ld, bool vec, uint32_t rows, uint32_t cols,
                                           uint32_t row0, uint32_t col0, uint32_t buf) {
    const uint32_t lane = threadIdx.x & 31;
    if (vec) {
#pragma unroll
        for (uint32_t i = lane; i < 4 * 32; i += 32) {
            const uint32_t r = i / 4, j = i % 4, col = col0 + 8 * j;
            if (row0 + r >= rows || col >= cols) continue;
            unsigned short* out = dst + static_cast<uint64_t>(row0 + r) * ld + col;
            const uint4 x = ld_shared(buf + piece64(r, j));
            if (col + 8 <= cols) {
                *reinterpret_cast<uint4*>(out) = x;
            } else {
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (uint32_t e = 0; e < 8; ++e)
                    if (col + e < cols) out[e] = static_cast<unsigned short>(w[e >> 1] >> (16 * (e & 1)));
            }
        }
    } else {
#pragma unroll 4
        for (uint32_t i = lane; i < 32 * 32; i += 32) {
            const uint32_t r = i / 32, e = i % 32;
            if (row0 + r < rows && col0 + e < cols)
                dst[static_cast<uint64_t>(row0 + r) * ld + col0 + e] =
                    ld_shared16(buf + piece64(r, e >> 3) + 2 * (e & 7));
        }
    }
}

// Lower-triangular tile t of a square grid of tiles: row i >= column j.
__device__ __forceinline__ void triangle(uint32_t t, uint32_t& i, uint32_t& j) {
    uint32_t r = static_cast<uint32_t>((__fsqrt_rn(8.0f * static_cast<float>(t) + 1.0f) - 1.0f) * 0.5f);
    while (r * (r + 1) / 2 > t) --r;
    while ((r + 1) * (r + 2) / 2 <= t) ++r;
    i = r;
    j = t - r * (r + 1) / 2;
}

// -------------------------------------------------------------------- host
inline cudaError_t sm_count(int* out) {
    static std::mutex mu;
    static int sms[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!sms[dev] && (e = cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
        return e;
    *out = sms[dev];
    return cudaSuccess;
}

// Raises a kernel's shared-memory limit, once per kernel and device.
template <auto Kernel>
cudaError_t allow_smem(size_t bytes) {
    static std::mutex mu;
    static uint64_t seen = 0;   // one bit a device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if ((seen >> dev) & 1) return cudaSuccess;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (e == cudaSuccess) seen |= 1ull << dev;
    return e;
}

// Reads this file's give-up word and, when it is set, clears it.
// Synchronises the stream.
inline cudaError_t read_gave_up(cudaStream_t s, int32_t* out) {
    static const int32_t zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(out, g_gave_up, sizeof(zero), 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess && *out)
        e = cudaMemcpyToSymbolAsync(g_gave_up, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s);
    return e;
}

}  // namespace
}  // namespace zg
