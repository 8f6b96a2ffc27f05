// The embedding of a training step: rows of a 16-bit table by token, and the
// table's gradient.
//
//   out[t] = s E[id_t];   dE[v] = s (sum over t with id_t = v of dy[t])
//
// Both move rows and are bound by HBM, the gradient mostly by writing the
// table: every row of it, most of them zeros.  Its sums are made without
// atomics on values, so that they do not depend on an order of arrival:
//
//   sort   the tokens by id, stably, by one cluster of 8 CTAs (radix digits
//          of up to 8 bits; its CTAs see each other's counts through their
//          shared memory, hand each other up to 16384 keys the same way, and
//          wait for each other at the cluster's barrier only).  The launch's
//          other CTAs fill the table with zeros meanwhile, which takes about
//          as long for some 8000 tokens and a table of a real size (both
//          together 14.6 us of which the 77 MB of zeros are 12 to 13).
//          Past 16384 tokens the keys go through global memory, and the sort
//          is what takes long.
//   sum    a warp takes 256 columns of kPiece consecutive sorted tokens, in
//          fp32.  A run of one id that lies inside its piece is finished and
//          written; one that crosses into other pieces leaves partial sums.
//   join   the warp of the piece in which such a run begins adds them in
//          order, or its block where there are many.
//
// Up to 512 tokens are not sorted: each looks at all ids (k_embedding_few).
// 8192 x 768 bf16 into 50257 rows takes 26.6 us, 6007 x 1003 fp16 into 32003
// 27.3: writing the table at the 6 TB/s that stores alone reach is 12 to 13 of
// them, all of the sort but some 2 hides behind it, and sum and join are
// chains of dependent reads, 12 us together, that nothing is left to hide.
// 65536 x 768 takes 88 to 91, 16384 x 4096 into 32000 92; with accumulate
// 8192 x 768 24, 65536 x 768 96.  (Partial sums added by
// the last warp of their run to come, with counters and fences in place of the
// join's launch: 27.4 and 32.2 us.)
//
// An id outside the table is padding: zeros forward, no gradient.

#include <cmath>
#include <cstdint>
#include <string>

#include <nvtx3/nvToolsExt.h>

#include "zero_gb300.h"
#include "zero_rows.cuh"
#include "zero_tc.cuh"

namespace zg {
namespace {

struct EmbedArgs {
    const unsigned short* table;
    unsigned short* out;
    const void* ids;
    uint64_t vocab, dim, tokens, ld_table, ld_out;
    uint64_t segments;   // of 256 columns
    float scale;
    int wide_ids;        // 8 bytes each, else 4
};

// The id of token t, or vocab for one outside the table.
__device__ __forceinline__ uint32_t id_at(const void* ids, int wide, uint64_t t, uint64_t vocab) {
    const int64_t id = wide ? static_cast<const int64_t*>(ids)[t] : static_cast<const int32_t*>(ids)[t];
    return id >= 0 && static_cast<uint64_t>(id) < vocab ? static_cast<uint32_t>(id) : static_cast<uint32_t>(vocab);
}

// A warp takes 256 columns of kEmbedTokens tokens, 8 a lane, all loads in
// flight together.
constexpr int kEmbedTokens = 4;

template <int DT, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) k_embedding(const __grid_constant__ EmbedArgs a) {
    pdl_enter();
    const uint64_t item = static_cast<uint64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    const uint64_t quad = item / a.segments, t0 = quad * kEmbedTokens;
    if (t0 >= a.tokens) return;
    const uint64_t c = (item - quad * a.segments) * 256;
    const int left = columns_left(a.dim, c);
    Loaded<ALIGNED> f[kEmbedTokens];
    uint32_t id[kEmbedTokens];
#pragma unroll
    for (int i = 0; i < kEmbedTokens; ++i) id[i] = t0 + i < a.tokens ? id_at(a.ids, a.wide_ids, t0 + i, a.vocab) : 0xFFFFFFFFu;
#pragma unroll
    for (int i = 0; i < kEmbedTokens; ++i)
        load_eight(a.table + (id[i] < a.vocab ? id[i] * a.ld_table + c : 0u), id[i] < a.vocab ? left : 0, f[i]);
#pragma unroll
    for (int i = 0; i < kEmbedTokens; ++i) {
        if (t0 + i >= a.tokens) break;
        float x[8];
        widen_eight<DT>(f[i], x);
        mul8(x, a.scale);
        uint32_t q[4];
        narrow8<DT>(x, q);
        store_eight<ALIGNED>(a.out + (t0 + i) * a.ld_out + c, left, q);
    }
}

// -------------------------------------------------------------------- sort
constexpr uint32_t kSortCtas = 8, kSortThreads = 1024, kDigits = 256, kMostPer = 4, kHere = 2048;

struct SortArgs {
    const void* ids;
    uint64_t vocab, tokens;
    int wide_ids;
    uint32_t passes, digit_bits;
    uint32_t *key[2], *index[2];   // the sorted ones end in [(passes - 1) & 1]
    // what the other CTAs fill with zeros: rows, or one range
    unsigned short* zero;
    uint64_t zero_rows, zero_cols, zero_ld;
};

__device__ __forceinline__ uint32_t load_of_cta(const uint32_t* shared, uint32_t cta) {
    uint32_t x;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(cluster_addr(smem_u32(shared), cta)) : "memory");
    return x;
}
__device__ __forceinline__ void store_to_cta(uint2* shared, uint32_t cta, uint2 x) {
    asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(cluster_addr(smem_u32(shared), cta)), "r"(x.x), "r"(x.y) : "memory");
}
// The cluster's barrier without waiting for this CTA's writes to global memory.
__device__ __forceinline__ void cluster_leave() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// What other CTAs of the cluster wrote comes from L2, not from this SM's L1.
__device__ __forceinline__ uint32_t load_l2(const uint32_t* p) {
    uint32_t x;
    asm volatile("ld.global.cg.u32 %0, [%1];" : "=r"(x) : "l"(p) : "memory");
    return x;
}

constexpr uint32_t kZeroBytes = 16384;

// By CTA `cta` of `ctas`.  Rows without gaps are one range, which a thread a
// CTA fills by bulk copies of `zeros` (77 MB in 12 to 13 us, 16-byte stores of
// all threads 18); rows with gaps a warp each.
__device__ void fill_zeros(const SortArgs& a, uint4 (&zeros)[kZeroBytes / 16], uint32_t cta, uint32_t ctas) {
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (a.zero_rows == 1) {
        for (uint32_t i = threadIdx.x; i < kZeroBytes / 16; i += kSortThreads) zeros[i] = make_uint4(0u, 0u, 0u, 0u);
        proxy_fence_shared();
        __syncthreads();
        uint64_t head = (16 - (reinterpret_cast<uintptr_t>(a.zero) & 15)) / 2 % 8;
        if (head > a.zero_cols) head = a.zero_cols;
        const uint64_t body = (a.zero_cols - head) / 8 * 16, done = head + body / 2;   // bytes of whole pieces
        if (warp == 1 && cta == 0) {
            if (lane < head) a.zero[lane] = 0;
            if (lane < a.zero_cols - done) a.zero[done + lane] = 0;
        }
        if (threadIdx.x != 0) return;
        unsigned char* to = reinterpret_cast<unsigned char*>(a.zero + head);
        for (uint64_t at = static_cast<uint64_t>(cta) * kZeroBytes; at < body; at += static_cast<uint64_t>(ctas) * kZeroBytes) {
            const uint32_t n = body - at < kZeroBytes ? static_cast<uint32_t>(body - at) : kZeroBytes;
            asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;"
                         ::"l"(to + at), "r"(smem_u32(zeros)), "r"(n)
                         : "memory");
        }
        store_commit();
        store_wait<0>();
        return;
    }
    for (uint64_t r = static_cast<uint64_t>(cta) * 32 + warp; r < a.zero_rows; r += static_cast<uint64_t>(ctas) * 32) {
        unsigned short* row = a.zero + r * a.zero_ld;
        uint64_t head = (16 - (reinterpret_cast<uintptr_t>(row) & 15)) / 2 % 8;
        if (head > a.zero_cols) head = a.zero_cols;
        const uint64_t pieces = (a.zero_cols - head) / 8, done = head + 8 * pieces;
        if (lane < head) row[lane] = 0;
        for (uint64_t i = lane; i < pieces; i += 32) reinterpret_cast<uint4*>(row + head)[i] = make_uint4(0u, 0u, 0u, 0u);
        if (lane < a.zero_cols - done) row[done + lane] = 0;
    }
}

__global__ void __launch_bounds__(kSortThreads) k_embedding_sort(const __grid_constant__ SortArgs a) {
    pdl_enter();
    constexpr uint32_t kWarps = kSortThreads / 32;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __shared__ __align__(128) uint4 s_zeros[kZeroBytes / 16];
    if (blockIdx.x >= kSortCtas) {
        fill_zeros(a, s_zeros, blockIdx.x - kSortCtas, gridDim.x - kSortCtas);
        return;
    }
    // a tile's keys of each digit, by warp; then those in the warps before
    unsigned short (*const s_warp)[kDigits] = reinterpret_cast<unsigned short (*)[kDigits]>(s_zeros);
    static_assert(sizeof(s_zeros) == kWarps * kDigits * sizeof(unsigned short) && kDigits * 4 == kSortThreads, "one place");
    __shared__ uint2 s_next[kHere];         // the next pass's keys and indexes, where the CTAs can hold them
    __shared__ uint32_t s_part[4][kDigits]; // a quarter of the warps' keys of each digit
    __shared__ uint32_t s_count[kDigits];   // this CTA's keys of each digit
    __shared__ uint32_t s_base[kDigits];    // where the tile's first key of a digit goes
    __shared__ uint32_t s_total[kDigits];   // the tile's keys of each digit
    __shared__ uint32_t s_scan[kDigits / 32];
    const uint32_t me = cluster_rank();
    const uint64_t share = (a.tokens + kSortCtas - 1) / kSortCtas, first = me * share;
    const uint64_t end = first >= a.tokens ? first : first + share < a.tokens ? first + share : a.tokens;
    // keys a thread has of a tile; a warp's are consecutive, 32 at a time
    const uint32_t per = share > 2 * kSortThreads ? kMostPer : share > kSortThreads ? 2 : 1, tile_keys = per * kSortThreads;
    const uint32_t digits = 1u << a.digit_bits;
    for (uint32_t pass = 0; pass < a.passes; ++pass) {
        const uint32_t shift = pass * a.digit_bits;
        const uint32_t* from = a.key[(pass & 1) ^ 1];
        const uint32_t* from_index = a.index[(pass & 1) ^ 1];
        uint32_t *to = a.key[pass & 1], *to_index = a.index[pass & 1];
        auto key_of = [&](uint64_t i) { return pass == 0 ? id_at(a.ids, a.wide_ids, i, a.vocab) : load_l2(from + i); };
        const bool one_tile = share <= tile_keys;   // then the tile's counts are the CTA's
        const bool here = share <= kHere;           // a place goes to the CTA whose keys it is among in the next pass
        const bool last = pass + 1 == a.passes;
        if (!one_tile) {
            if (threadIdx.x < kDigits) s_count[threadIdx.x] = 0;
            __syncthreads();
#pragma unroll 4
            for (uint64_t i = first + threadIdx.x; i < end; i += kSortThreads)
                atomicAdd(&s_count[(key_of(i) >> shift) & (digits - 1)], 1u);
        }
        uint64_t tile = first;
        bool placed = false;   // s_base is set
        do {
            uint32_t key[kMostPer], index[kMostPer], rank[kMostPer];
            const uint64_t mine = tile + warp * (32 * per) + lane;
#pragma unroll
            for (uint32_t k = 0; k < kMostPer; ++k) {
                const uint64_t i = mine + 32 * k;
                if (k >= per || i >= end) continue;
                if (pass == 0 || !here) {
                    key[k] = key_of(i);
                    index[k] = pass == 0 ? static_cast<uint32_t>(i) : load_l2(from_index + i);
                } else {
                    const uint2 x = s_next[i - first];
                    key[k] = x.x;
                    index[k] = x.y;
                }
            }
            s_zeros[threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
            __syncthreads();
#pragma unroll
            for (uint32_t k = 0; k < kMostPer; ++k) {   // the keys of the same digit before this one in the warp
                if (k >= per) break;
                const bool some = mine + 32 * k < end;
                const uint32_t digit = some ? (key[k] >> shift) & (digits - 1) : kDigits;
                const uint32_t same = __match_any_sync(0xFFFFFFFFu, digit), ahead = __popc(same & ((1u << lane) - 1));
                const uint32_t so_far = some ? s_warp[warp][digit] : 0u;
                rank[k] = so_far + ahead;
                __syncwarp();
                if (some && ahead == 0) s_warp[warp][digit] = static_cast<unsigned short>(so_far + __popc(same));
                __syncwarp();
            }
            __syncthreads();
            {   // four threads a digit, 8 warps each
                constexpr uint32_t kEach = kWarps / 4;
                const uint32_t digit = threadIdx.x & (kDigits - 1), part = threadIdx.x / kDigits;
                uint32_t n[kEach], sum = 0;
#pragma unroll
                for (uint32_t q = 0; q < kEach; ++q) n[q] = s_warp[part * kEach + q][digit];
#pragma unroll
                for (uint32_t q = 0; q < kEach; ++q) {
                    const uint32_t x = n[q];
                    n[q] = sum;
                    sum += x;
                }
                s_part[part][digit] = sum;
                __syncthreads();
                uint32_t before = 0;
                for (uint32_t q = 0; q < part; ++q) before += s_part[q][digit];
                if (part == 3) {
                    s_total[digit] = before + sum;
                    if (one_tile) s_count[digit] = before + sum;
                }
#pragma unroll
                for (uint32_t q = 0; q < kEach; ++q)
                    s_warp[part * kEach + q][digit] = static_cast<unsigned short>(n[q] + before);
            }
            if (!placed) {   // the CTAs' counts are complete
                cluster_sync();
                // keys of smaller digits anywhere, and of the same digit in the CTAs before
                uint32_t base = 0;
                if (threadIdx.x < kDigits) {
                    uint32_t all = 0;
#pragma unroll
                    for (uint32_t q = 0; q < kSortCtas; ++q) {
                        const uint32_t n = load_of_cta(&s_count[threadIdx.x], q);
                        base += q < me ? n : 0u;
                        all += n;
                    }
                    uint32_t sum = all;   // inclusive scan over the digits
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) {
                        const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, sum, d);
                        if (lane >= static_cast<uint32_t>(d)) sum += x;
                    }
                    if (lane == 31) s_scan[warp] = sum;
                    base += sum - all;
                }
                __syncthreads();
                if (threadIdx.x < kDigits) {
                    for (uint32_t q = 0; q < warp; ++q) base += s_scan[q];
                    s_base[threadIdx.x] = base;
                }
                placed = true;
            }
            __syncthreads();
#pragma unroll
            for (uint32_t k = 0; k < kMostPer; ++k) {
                if (k >= per || mine + 32 * k >= end) continue;
                const uint32_t digit = (key[k] >> shift) & (digits - 1);
                const uint32_t at = s_base[digit] + s_warp[warp][digit] + rank[k];
                if (here && !last) {
                    const uint32_t cta = at / static_cast<uint32_t>(share);
                    store_to_cta(&s_next[at - cta * static_cast<uint32_t>(share)], cta, make_uint2(key[k], index[k]));
                } else {
                    to[at] = key[k];
                    to_index[at] = index[k];
                }
            }
            tile += tile_keys;
            if (one_tile || tile >= end) break;
            __syncthreads();
            if (threadIdx.x < kDigits) s_base[threadIdx.x] += s_total[threadIdx.x];
        } while (true);
        if (last) cluster_leave();   // the other CTAs have read its counts
        else cluster_sync();
    }
}

// The zeros by themselves.
__global__ void __launch_bounds__(kSortThreads) k_embedding_zeros(const __grid_constant__ SortArgs a) {
    pdl_enter();
    __shared__ __align__(128) uint4 s_zeros[kZeroBytes / 16];
    fill_zeros(a, s_zeros, blockIdx.x, gridDim.x);
}

// -------------------------------------------------------------- sum and join
struct SumArgs {
    const unsigned short* grad;
    unsigned short* table;
    const uint32_t *key, *index;   // sorted tokens
    float* partial;                // [pieces][2][8 * across]: of the run that enters a piece, of the one that leaves it
    uint64_t vocab, dim, tokens, ld_grad, ld_table;
    uint64_t segments, pieces, width;   // width = 8 * ceil(dim / 8)
    float scale;
    int add;                       // to what the table holds
};
constexpr uint32_t kPiece = 8;

// A warp's 256 columns from c on, `left` of them inside the row: a sum, times
// the factor, into its row of the table.
template <int DT, bool ALIGNED>
__device__ __forceinline__ void write_sum(const SumArgs& a, uint32_t id, uint64_t c, int left, float (&s)[8]) {
    unsigned short* at = a.table + id * a.ld_table + c;
    mul8(s, a.scale);
    if (a.add) {
        Loaded<ALIGNED> r;
        load_eight(at, left, r);
        float x[8];
        widen_eight<DT>(r, x);
        add8(s, x);
    }
    uint32_t q[4];
    narrow8<DT>(s, q);
    store_eight<ALIGNED>(at, left, q);
}
__device__ __forceinline__ float* partial_at(const SumArgs& a, uint64_t piece, int leaves, uint64_t c) {
    return a.partial + (2 * piece + leaves) * a.width + c;
}
// A warp's 256 values in shared memory.
__device__ __forceinline__ void put_shared(uint4* at, const Loaded<true>& r) { at[threadIdx.x & 31] = r.x; }
__device__ __forceinline__ void get_shared(const uint4* at, Loaded<true>& r) { r.x = at[threadIdx.x & 31]; }
__device__ __forceinline__ void put_shared(uint4* at, const Loaded<false>& r) {
#pragma unroll
    for (int e = 0; e < 8; ++e) reinterpret_cast<unsigned short*>(at)[column_of<false>(e)] = r.x[e];
}
__device__ __forceinline__ void get_shared(const uint4* at, Loaded<false>& r) {
#pragma unroll
    for (int e = 0; e < 8; ++e) r.x[e] = reinterpret_cast<const unsigned short*>(at)[column_of<false>(e)];
}
template <bool ALIGNED>
__device__ __forceinline__ void write_partial(float* at, int left, const float (&s)[8]) {
    if constexpr (ALIGNED) {
        if (static_cast<int>(column_of<true>(0)) >= left) return;
        float4* to = reinterpret_cast<float4*>(at + column_of<true>(0));
        to[0] = make_float4(s[0], s[1], s[2], s[3]);
        to[1] = make_float4(s[4], s[5], s[6], s[7]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (static_cast<int>(column_of<false>(e)) < left) at[column_of<false>(e)] = s[e];
    }
}
template <bool ALIGNED>
__device__ __forceinline__ void add_partial(const float* at, int left, float (&s)[8]) {
    float x[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (ALIGNED) {
        if (static_cast<int>(column_of<true>(0)) < left) {
            const float4* from = reinterpret_cast<const float4*>(at + column_of<true>(0));
            const float4 y = from[0], z = from[1];
            x[0] = y.x; x[1] = y.y; x[2] = y.z; x[3] = y.w;
            x[4] = z.x; x[5] = z.y; x[6] = z.z; x[7] = z.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (static_cast<int>(column_of<false>(e)) < left) x[e] = at[column_of<false>(e)];
    }
    add8(s, x);
}

template <int DT, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 3) k_embedding_sum(const __grid_constant__ SumArgs a) {
    pdl_enter();
    __shared__ uint4 s_rows[kThreads / 32][kPiece][32];   // 256 values each
    const uint64_t item = static_cast<uint64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    const uint64_t piece = item / a.segments;
    if (piece >= a.pieces) return;
    const uint32_t lane = threadIdx.x & 31;
    const uint64_t c = (item - piece * a.segments) * 256, first = piece * kPiece;
    const int left = columns_left(a.dim, c);
    const uint32_t none = static_cast<uint32_t>(a.vocab);   // padding, sorted behind all ids
    // lane i: the piece's token i; lanes 30 and 31 the neighbours' ids
    const uint64_t mine = lane == 30 ? first - 1 : lane == 31 ? first + kPiece : first + lane;
    const bool there = lane == 30 ? first > 0 : mine < a.tokens && (lane == 31 || lane < kPiece);
    const uint32_t key = there ? load_l2(a.key + mine) : none;
    const uint32_t index = there && lane < kPiece ? load_l2(a.index + mine) : 0u;
    const uint32_t before = __shfl_sync(0xFFFFFFFFu, key, 30), after = __shfl_sync(0xFFFFFFFFu, key, 31);
    const uint32_t count = __popc(__ballot_sync(0xFFFFFFFFu, lane < kPiece && key != none));
    if (count == 0) return;
    // all rows in flight together; then one after the other in a loop, through
    // shared memory, of which every lane reads what it wrote: a short loop's
    // instructions are there sooner than those of eight copies
    uint4 (*const rows)[32] = s_rows[threadIdx.x >> 5];
    {
        Loaded<ALIGNED> f[kPiece];
#pragma unroll
        for (uint32_t i = 0; i < kPiece; ++i)
            load_eight(a.grad + __shfl_sync(0xFFFFFFFFu, index, i) * a.ld_grad + c, i < count ? left : 0, f[i]);
#pragma unroll
        for (uint32_t i = 0; i < kPiece; ++i) put_shared(rows[i], f[i]);
    }
    float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    uint32_t id = __shfl_sync(0xFFFFFFFFu, key, 0);
    bool enters = first > 0 && id == before;   // the run began in an earlier piece
#pragma unroll 1
    for (uint32_t i = 0; i < count; ++i) {
        float y[8];
        Loaded<ALIGNED> x;
        get_shared(rows[i], x);
        widen_eight<DT>(x, y);
        add8(s, y);
        const uint32_t next = i + 1 < count ? __shfl_sync(0xFFFFFFFFu, key, i + 1) : count == kPiece ? after : none;
        if (next == id && i + 1 < count) continue;
        // the run is complete here, or leaves the piece
        if (enters || next == id) write_partial<ALIGNED>(partial_at(a, piece, enters ? 0 : 1, c), left, s);
        else write_sum<DT, ALIGNED>(a, id, c, left, s);
        id = next;
        enters = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = 0.0f;
    }
}

// A block looks at kJoinPieces pieces, a warp each, for a run that begins in
// the piece and goes on in the next one, and adds its partial sums of 256
// columns.  A warp adds a run over up to kShortRun pieces by itself; the
// block's warps share the others (the frequent tokens of a language model's
// batch cover some ten pieces each), every eighth piece a warp, and add their
// sums in order.
constexpr uint32_t kJoinPieces = kThreads / 32, kShortRun = 8;

template <int DT, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) k_embedding_join(const __grid_constant__ SumArgs a) {
    pdl_enter();
    __shared__ uint32_t s_id[kJoinPieces], s_run[kJoinPieces];   // a long run that begins in the warp's piece, or none (0)
    __shared__ __align__(16) float s_sum[kJoinPieces][256];
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t group = blockIdx.x / a.segments, piece = group * kJoinPieces + warp;
    const uint64_t c = (blockIdx.x - group * a.segments) * 256;
    const int left = columns_left(a.dim, c);
    auto add = [&](float (&s)[8], uint64_t p, int leaves) { add_partial<ALIGNED>(partial_at(a, p, leaves, c), left, s); };
    uint32_t id = 0, run = 0;   // the pieces after this one that the run enters
    const uint64_t first = piece * kPiece;
    if (piece + 1 < a.pieces) {
        const uint32_t none = static_cast<uint32_t>(a.vocab);
        id = load_l2(a.key + first + kPiece - 1);
        const uint32_t before = first > 0 ? load_l2(a.key + first - 1) : none;
        const uint64_t q = piece + 1 + lane, rest = a.pieces - piece - 1;
        const uint32_t next = q < a.pieces ? load_l2(a.key + q * kPiece) : none;
        // a run that fills the whole piece (the ids are sorted) may have begun earlier
        if (id < none && before != id) {
            const uint32_t in = __ballot_sync(0xFFFFFFFFu, next == id);
            run = in == 0xFFFFFFFFu ? 32u : __ffs(~in) - 1;
            if (run == 32u) {   // a long one: its end is in (low, high]; 32 places of that at a time
                uint64_t low = 31, high = rest;
                while (high - low > 1) {
                    const uint64_t step = (high - low + 31) / 32, at = low + (lane + 1) * step;
                    const uint32_t still = __ballot_sync(0xFFFFFFFFu, at < high && load_l2(a.key + (piece + 1 + at) * kPiece) == id);
                    const uint32_t n = still == 0xFFFFFFFFu ? 32u : __ffs(~still) - 1;   // sorted: the first n are in the run
                    const uint64_t to = low + (n + 1) * step;
                    low += n * step;
                    high = to < high ? to : high;
                }
                run = static_cast<uint32_t>(high);
            }
        }
    }
    float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (lane == 0) {
        s_id[warp] = id;
        s_run[warp] = run > kShortRun ? run : 0;
    }
    if (run > 0 && run <= kShortRun) {
        add(s, piece, 1);
#pragma unroll
        for (uint32_t i = 0; i < kShortRun; ++i)
            if (i < run) add(s, piece + 1 + i, 0);
        write_sum<DT, ALIGNED>(a, id, c, left, s);
    }
    __syncthreads();
    for (uint32_t k = 0; k < kJoinPieces; ++k) {
        const uint32_t pieces = s_run[k];
        if (pieces == 0) continue;   // the same for all
        const uint64_t from = group * kJoinPieces + k;
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = 0.0f;
        if (warp == 0) add(s, from, 1);
#pragma unroll 8
        for (uint32_t i = warp; i < pieces; i += kJoinPieces) add(s, from + 1 + i, 0);
#pragma unroll
        for (int e = 0; e < 8; ++e) s_sum[warp][32 * e + lane] = s[e];
        __syncthreads();
        if (warp == 0) {
#pragma unroll
            for (uint32_t w = 1; w < kJoinPieces; ++w) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = s_sum[w][32 * e + lane];
                add8(s, x);
            }
            write_sum<DT, ALIGNED>(a, s_id[k], c, left, s);
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------ few tokens
// Up to kFewTokens tokens need no sorting: a block takes 256 columns of one
// token, looks at all ids, and leaves where the token's own occurs before.
// Else it adds up the rows with that id: each warp those of every eighth
// token, in order, then the warps' sums in order.  So a run of one id (a
// batch whose padding is a row of the table) is read by eight warps, each
// with as many rows in flight as its registers allow at full occupancy: with
// accumulate 512 tokens of 768 columns take 4.7 us by Zipf's law and 11.3
// with one id (sorted: 14.8 and 13.7; one warp a run: 9.4 and 71).  Six rows
// against four and eight: 512 of one id 28.5 us (32.9, 25.6), 512 x 4096 by
// Zipf's law with accumulate 14.3 (12.8, 16.1).
struct FewArgs {
    SumArgs sum;
    const void* ids;
    int wide_ids;
};
constexpr uint32_t kFewTokens = 512;

template <int DT, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) k_embedding_few(const __grid_constant__ FewArgs f) {
    pdl_enter();
    constexpr uint32_t kWarps = kThreads / 32, kLooks = kFewTokens / kThreads, kAhead = ALIGNED ? 6 : 4;
    static_assert(kFewTokens % kThreads == 0, "a thread looks at kLooks ids");
    __shared__ uint32_t s_some[kWarps];
    __shared__ float s_sum[kWarps][256];
    const SumArgs& a = f.sum;
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tokens = static_cast<uint32_t>(a.tokens);
    const uint32_t segments = static_cast<uint32_t>(a.segments), t = blockIdx.x / segments;
    const uint32_t none = static_cast<uint32_t>(a.vocab), id = id_at(f.ids, f.wide_ids, t, a.vocab);
    uint32_t same[kLooks];   // bit l: token kThreads k + kWarps l + warp has this id
    bool before = false;
#pragma unroll
    for (uint32_t k = 0; k < kLooks; ++k) {
        const uint32_t i = kThreads * k + kWarps * lane + warp;
        const bool is = i < tokens && id_at(f.ids, f.wide_ids, i, a.vocab) == id;
        same[k] = __ballot_sync(0xFFFFFFFFu, is);
        before = before || (is && i < t);
    }
    if (lane == 0) {
        uint32_t some = 0;
#pragma unroll
        for (uint32_t k = 0; k < kLooks; ++k) some |= same[k];
        s_some[warp] = some;
    }
    if (__syncthreads_or(before) || id == none) return;
    const uint32_t warps = __ballot_sync(0xFFFFFFFFu, lane < kWarps && s_some[lane % kWarps] != 0);   // those that have rows
    const bool alone = (warps & (warps - 1)) == 0;
    if (alone && warps != 1u << warp) return;
    const uint64_t c = static_cast<uint64_t>(blockIdx.x - t * segments) * 256;
    const int left = columns_left(a.dim, c);
    float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
    for (uint32_t k = 0; k < kLooks; ++k) {
        uint32_t rest = same[0];
#pragma unroll
        for (uint32_t q = 1; q < kLooks; ++q) rest = k == q ? same[q] : rest;
#pragma unroll 1
        while (rest) {   // kAhead rows in flight
            Loaded<ALIGNED> r[kAhead];
#pragma unroll
            for (uint32_t i = 0; i < kAhead; ++i) {
                const uint64_t at = kThreads * k + kWarps * (rest ? __ffs(rest) - 1 : 0) + warp;
                load_eight(a.grad + at * a.ld_grad + c, rest ? left : 0, r[i]);
                rest &= rest - 1;
            }
#pragma unroll
            for (uint32_t i = 0; i < kAhead; ++i) {
                float x[8];
                widen_eight<DT>(r[i], x);
                add8(s, x);
            }
        }
    }
    if (!alone) {
#pragma unroll
        for (int e = 0; e < 8; ++e) s_sum[warp][32 * e + lane] = s[e];
        __syncthreads();
        if (warp + 1 != __ffs(warps)) return;
#pragma unroll 1
        for (uint32_t rest = warps & (warps - 1); rest; rest &= rest - 1) {
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = s_sum[__ffs(rest) - 1][32 * e + lane];
            add8(s, x);
        }
    }
    write_sum<DT, ALIGNED>(a, id, c, left, s);
}

// -------------------------------------------------------------------- host
constexpr uint64_t kMaxTokens = 1ull << 31, kMaxVocab = 1ull << 31, kMaxDim = 1ull << 20, kMaxLd = 1ull << 40;

int check_embedding(int dtype, uint64_t vocab, uint64_t dim, uint64_t tokens, const void* ids, int id_bytes, float scale) {
    if (dtype != ZERO_FP16 && dtype != ZERO_BF16) return refuse(ZERO_EINVAL, "dtype must be fp16 or bf16");
    if (vocab < 1 || vocab > kMaxVocab) return refuse(ZERO_EINVAL, "vocab must be in 1..2^31");
    if (dim > kMaxDim) return refuse(ZERO_EINVAL, "dim is more than 2^20");
    if (tokens > kMaxTokens) return refuse(ZERO_EINVAL, "more than 2^31 tokens");
    if (id_bytes != 4 && id_bytes != 8) return refuse(ZERO_EINVAL, "id_bytes must be 4 or 8");
    if (!std::isfinite(scale)) return refuse(ZERO_EINVAL, "scale must be finite");
    if (tokens && dim && (!ids || !aligned(ids, static_cast<uintptr_t>(id_bytes))))
        return refuse(ZERO_EINVAL, "ids is NULL or not aligned to its elements");
    return ZERO_OK;
}
int check_rows(const char* name, const void* at, uint64_t ld, uint64_t dim) {
    if (!at || !aligned(at, 2)) return refuse(ZERO_EINVAL, std::string(name) + " is NULL or not 2-byte aligned");
    if (ld < dim || ld > kMaxLd)
        return refuse(ZERO_EINVAL, "ld of " + std::string(name) + " must be at least dim (and at most 2^40)");
    return ZERO_OK;
}
constexpr uint64_t kZeroCtas = 304;   // two an SM
uint64_t sort_bytes(uint64_t tokens) { return up(tokens * 4, 256); }   // one of four arrays
uint64_t pieces_of(uint64_t tokens) { return (tokens + kPiece - 1) / kPiece; }

}  // namespace
}  // namespace zg

using namespace zg;

extern "C" {

int zero_embedding(int dtype, uint64_t vocab, uint64_t dim, const void* table16, uint64_t ld_table, uint64_t tokens,
                   const void* ids, int id_bytes, float scale, void* out16, uint64_t ld_out, void* stream) {
    nvtxRangePushA("zero_embedding");
    struct Pop { ~Pop() { nvtxRangePop(); } } pop;
    if (const int rc = check_embedding(dtype, vocab, dim, tokens, ids, id_bytes, scale)) return rc;
    if (tokens == 0 || dim == 0) return ZERO_OK;
    if (const int rc = check_rows("table16", table16, ld_table, dim)) return rc;
    if (const int rc = check_rows("out16", out16, ld_out, dim)) return rc;
    EmbedArgs a = {};
    a.table = static_cast<const unsigned short*>(table16);
    a.out = static_cast<unsigned short*>(out16);
    a.ids = ids;
    a.vocab = vocab;
    a.dim = dim;
    a.tokens = tokens;
    a.ld_table = ld_table;
    a.ld_out = ld_out;
    a.segments = up(dim, 256) / 256;
    a.scale = scale;
    a.wide_ids = id_bytes == 8;
    const uint64_t items = up(tokens, kEmbedTokens) / kEmbedTokens * a.segments, blocks = up(items, kThreads / 32) / (kThreads / 32);
    if (blocks > 0x7FFFFFFFull) return refuse(ZERO_EINVAL, "tokens and dim are too large together");
    const bool fp16 = dtype == ZERO_FP16;
    const bool whole = dim % 8 == 0 && aligned(table16, 16) && ld_table % 8 == 0 && aligned(out16, 16) && ld_out % 8 == 0;
    const cudaError_t e = launch_pdl(whole ? (fp16 ? k_embedding<kFp16, true> : k_embedding<kBf16, true>)
                                           : (fp16 ? k_embedding<kFp16, false> : k_embedding<kBf16, false>),
                                     dim3(static_cast<unsigned>(blocks)), kThreads, 0, 1, static_cast<cudaStream_t>(stream), a);
    return e == cudaSuccess ? ZERO_OK : cuda_refuse(e, "zero_embedding");
}

uint64_t zero_embedding_backward_workspace_bytes(uint64_t vocab, uint64_t dim, uint64_t tokens) {
    if (vocab < 1 || vocab > kMaxVocab || dim == 0 || dim > kMaxDim || tokens == 0 || tokens > kMaxTokens) return 0;
    return 4 * sort_bytes(tokens) + pieces_of(tokens) * 2 * up(dim, 8) * sizeof(float);
}

int zero_embedding_backward(int dtype, uint64_t vocab, uint64_t dim, const void* dout16, uint64_t ld_dout, uint64_t tokens,
                            const void* ids, int id_bytes, float scale, int accumulate, void* dtable16, uint64_t ld_dtable,
                            void* workspace, uint64_t workspace_bytes, void* stream) {
    nvtxRangePushA("zero_embedding_backward");
    struct Pop { ~Pop() { nvtxRangePop(); } } pop;
    if (const int rc = check_embedding(dtype, vocab, dim, tokens, ids, id_bytes, scale)) return rc;
    if (dim == 0) return ZERO_OK;
    if (const int rc = check_rows("dtable16", dtable16, ld_dtable, dim)) return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (tokens == 0) {   // empty sums
        e = accumulate ? cudaSuccess : cudaMemset2DAsync(dtable16, ld_dtable * 2, 0, dim * 2, vocab, s);
        return e == cudaSuccess ? ZERO_OK : cuda_refuse(e, "zero_embedding_backward");
    }
    if (const int rc = check_rows("dout16", dout16, ld_dout, dim)) return rc;
    if (!workspace || !aligned(workspace, 256)) return refuse(ZERO_EINVAL, "workspace is NULL or not 256-byte aligned");
    if (workspace_bytes < zero_embedding_backward_workspace_bytes(vocab, dim, tokens))
        return refuse(ZERO_EINVAL, "workspace is smaller than zero_embedding_backward_workspace_bytes()");
    const uint64_t segments = up(dim, 256) / 256;
    if (up(pieces_of(tokens), kThreads / 32) / (kThreads / 32) * segments > 0x7FFFFFFFull)
        return refuse(ZERO_EINVAL, "tokens and dim are too large together");
    unsigned char* at = static_cast<unsigned char*>(workspace);
    SortArgs o = {};
    o.ids = ids;
    o.vocab = vocab;
    o.tokens = tokens;
    o.wide_ids = id_bytes == 8;
    uint32_t bits = 1;
    while (vocab >> bits) ++bits;   // of the ids and of vocab itself, which stands for padding
    o.passes = (bits + 7) / 8;
    o.digit_bits = (bits + o.passes - 1) / o.passes;
    for (int i = 0; i < 2; ++i, at += 2 * sort_bytes(tokens)) {
        o.key[i] = reinterpret_cast<uint32_t*>(at);
        o.index[i] = reinterpret_cast<uint32_t*>(at + sort_bytes(tokens));
    }
    uint64_t others = 0;
    if (!accumulate) {
        o.zero = static_cast<unsigned short*>(dtable16);
        const bool range = ld_dtable == dim;
        o.zero_rows = range ? 1 : vocab;
        o.zero_cols = range ? vocab * dim : dim;
        o.zero_ld = ld_dtable;
        others = range ? up(2 * o.zero_cols, kZeroBytes) / kZeroBytes : up(vocab, 32) / 32;
        if (others > kZeroCtas) others = kZeroCtas;
    }
    FewArgs f = {};
    SumArgs& a = f.sum;
    a.grad = static_cast<const unsigned short*>(dout16);
    a.table = static_cast<unsigned short*>(dtable16);
    a.key = o.key[(o.passes - 1) & 1];
    a.index = o.index[(o.passes - 1) & 1];
    a.partial = reinterpret_cast<float*>(at);
    a.vocab = vocab;
    a.dim = dim;
    a.tokens = tokens;
    a.ld_grad = ld_dout;
    a.ld_table = ld_dtable;
    a.segments = segments;
    a.pieces = pieces_of(tokens);
    a.width = up(dim, 8);
    a.scale = scale;
    a.add = accumulate != 0;
    const bool fp16 = dtype == ZERO_FP16;
    const bool whole = dim % 8 == 0 && aligned(dout16, 16) && ld_dout % 8 == 0 && aligned(dtable16, 16) && ld_dtable % 8 == 0;
    constexpr unsigned kWarps = kThreads / 32;
    // without sorting (by Zipf's law, sorted in brackets): 128 tokens of 768 columns into 50257 rows 15.0 us (19.9), 512 16.7
    // (20.7), of 4096 into 32000 53.8 (51.4); one id for all of them 17.8 (20.2), 28.5 (22.2), 57.1 (52.9)
    if (tokens <= kFewTokens) {
        f.ids = ids;
        f.wide_ids = o.wide_ids;
        e = accumulate ? cudaSuccess
                       : launch_pdl(k_embedding_zeros, dim3(static_cast<unsigned>(others)), kSortThreads, 0, 1, s, o);
        if (e == cudaSuccess)
            e = launch_pdl(whole ? (fp16 ? k_embedding_few<kFp16, true> : k_embedding_few<kBf16, true>)
                                 : (fp16 ? k_embedding_few<kFp16, false> : k_embedding_few<kBf16, false>),
                           dim3(static_cast<unsigned>(tokens * segments)), kThreads, 0, 1, s, f);
        return e == cudaSuccess ? ZERO_OK : cuda_refuse(e, "zero_embedding_backward");
    }
    e = launch_pdl(k_embedding_sort, dim3(static_cast<unsigned>(kSortCtas + up(others, kSortCtas))), kSortThreads, 0, kSortCtas, s, o);
    if (e == cudaSuccess)
        e = launch_pdl(whole ? (fp16 ? k_embedding_sum<kFp16, true> : k_embedding_sum<kBf16, true>)
                             : (fp16 ? k_embedding_sum<kFp16, false> : k_embedding_sum<kBf16, false>),
                       dim3(static_cast<unsigned>((a.pieces * segments + kWarps - 1) / kWarps)), kThreads, 0, 1, s, a);
    if (e == cudaSuccess)
        e = launch_pdl(whole ? (fp16 ? k_embedding_join<kFp16, true> : k_embedding_join<kBf16, true>)
                             : (fp16 ? k_embedding_join<kFp16, false> : k_embedding_join<kBf16, false>),
                       dim3(static_cast<unsigned>(up(a.pieces, kJoinPieces) / kJoinPieces * segments)), kThreads, 0, 1, s, a);
    return e == cudaSuccess ? ZERO_OK : cuda_refuse(e, "zero_embedding_backward");
}

}  // extern "C"
