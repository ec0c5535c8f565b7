// The pages of a paged cache on the device: fork (children of a request share
// its full pages and get their own copy of the partial last one), release
// (references of a range of pages given back) and compaction (the live pages
// moved to the lowest ids).
//
// A page is live while its reference count is positive. Free pages are found by
// their rank: the k-th free page is the k-th lowest id with count 0, from per-chunk
// counts and a scan of one chunk, so no free list has to be kept and the result
// does not depend on the order in which blocks run. Counts are int32 atomics.
//
// All of it is bound by memory: the counts are read once (fork, compaction: by
// kernels of kChunk ids per block), the tables once, and every copied page once,
// with 16-byte vectors, several loads in flight per thread. Small calls are bound
// by their launches instead: where the counts and tables are small enough, the
// steps of a call up to the page copies run in one cluster of kCluster blocks, a
// cluster barrier between them, in place of a kernel each. Measured per call of a
// stream of them: fork and release of four beams over 2000 pages 23.8 -> 20.6 us,
// release and compaction of six requests over 600 pages 31 -> 20.9 us; but over
// 36000 pages and 65000 entries, where eight blocks are too few, 55 -> 65 us.
#include <cuda_runtime.h>
#include <stdint.h>

#include "abi_checks.h"
#include "pcp.h"
#include "pcp_device.cuh"
#include "pcp_internal.h"

namespace pcp {

namespace {

constexpr int kPageThreads = 256;
constexpr int kPer = 4;                           // ids per thread of a chunk
constexpr int kChunk = kPageThreads * kPer;       // ids per counting block
constexpr int kCopyThreads = 512;
constexpr int kCopyUnroll = 4;                    // 16-byte loads in flight per thread

constexpr int kCluster = 8;
constexpr int kClusterThreads = 1024;
constexpr int kClusterPer = 2;                    // ids per thread at most in a cluster's plan of moves
// the largest calls that take the one-cluster form
constexpr int64_t kClusterIds = (int64_t)kCluster * kClusterThreads * kClusterPer;
constexpr int64_t kClusterEntries = kClusterIds;
constexpr int32_t kClusterChildren = 16;

struct PagesLayout {
    size_t header, counts, holes, movers, rank, total;
    int32_t chunks;
};

PagesLayout pages_layout(int64_t num_blocks) {
    PagesLayout w{};
    w.chunks = (int32_t)((num_blocks + kChunk - 1) / kChunk);
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o = align256(o + bytes);
        return at;
    };
    w.header = take(64);
    w.counts = take((size_t)w.chunks * 4);
    w.holes = take((size_t)num_blocks * 4);
    w.movers = take((size_t)num_blocks * 4);
    w.rank = take((size_t)num_blocks * 4);
    w.total = o;
    return w;
}

// Sum of v over the block, to every thread.
template <int kThreads = kPageThreads>
__device__ __forceinline__ int32_t block_sum(int32_t v, int32_t* warp_sums) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();  // the previous use of warp_sums is over
    if (threadIdx.x % 32 == 0) warp_sums[threadIdx.x / 32] = v;
    __syncthreads();
    int32_t s = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) s += warp_sums[w];
    return s;
}

// Sum of v over the threads before this one.
__device__ __forceinline__ int32_t block_before(int32_t v, int32_t* warp_sums) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int32_t before = x - v;
    for (int w = 0; w < warp; ++w) before += warp_sums[w];
    return before;
}

// This thread's kPer consecutive ids of a chunk: bit e set where id e is live
// (positive count). Ids past the pool count as neither live nor free; *in_pool
// is the number of ids that exist.
__device__ __forceinline__ uint32_t live_bits(const int32_t* ref, int64_t id0, int64_t num_blocks, int* in_pool) {
    uint32_t bits = 0;
    int n = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e)
        if (id0 + e < num_blocks) {
            ++n;
            if (__ldg(ref + id0 + e) > 0) bits |= 1u << e;
        }
    *in_pool = n;
    return bits;
}

// counts[c] = free (kFree) or live ids of chunk c; ref_out, where given, becomes a
// copy of ref.
template <bool kFree>
__global__ void __launch_bounds__(kPageThreads)
    count_kernel(const int32_t* __restrict__ ref, int32_t* __restrict__ ref_out, int64_t num_blocks, int32_t* counts) {
    __shared__ int32_t warp_sums[kPageThreads / 32];
    const int64_t base = (int64_t)blockIdx.x * kChunk;
    int32_t n = 0;
    grid_launch_dependents();
    int32_t r[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const int64_t i = base + e * kPageThreads + threadIdx.x;
        r[e] = i < num_blocks ? ref[i] : 0;
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const int64_t i = base + e * kPageThreads + threadIdx.x;
        if (i >= num_blocks) continue;
        if (ref_out) ref_out[i] = r[e];
        n += (r[e] > 0) != kFree;
    }
    n = block_sum(n, warp_sums);
    if (threadIdx.x == 0) counts[blockIdx.x] = n;
}

struct ForkArgs {
    uint4 *kc, *vc;
    int64_t num_blocks;
    int32_t bs, vec_per_slot;
    const int32_t* table;
    int32_t num_reqs, mb;
    const int32_t *kv_len, *parent;
    int32_t children;
    const int32_t* ref;
    int32_t *table_out, *ref_out;
    int32_t* counts;  // free ids per chunk
    int32_t chunks;
    int32_t* status;
};

// One child, by a block of kPageThreads, once the counts are there.
__device__ __forceinline__ void fork_child(const ForkArgs& f, int32_t child, int32_t* warp_sums, int32_t& found) {
    const int64_t num_blocks = f.num_blocks;
    const int32_t bs = f.bs, vec_per_slot = f.vec_per_slot, num_reqs = f.num_reqs, mb = f.mb, chunks = f.chunks;
    const int32_t *table = f.table, *kv_len = f.kv_len, *parent = f.parent, *ref = f.ref, *counts = f.counts;
    int32_t *table_out = f.table_out, *ref_out = f.ref_out, *status = f.status;
    uint4 *kc = f.kc, *vc = f.vc;
    // tokens of child j: its parent's, 0 where it has none or a bad one
    auto tokens_of = [&](int32_t j) -> int32_t {
        const int32_t p = __ldg(parent + j);
        if (p < 0 || p >= num_reqs) return 0;
        const int32_t n = __ldg(kv_len + p);
        return n < 0 || n > (int64_t)mb * bs ? 0 : n;
    };
    const int32_t p = parent[child];
    const int32_t len = tokens_of(child);
    if (threadIdx.x == 0 && (p >= num_reqs || (p >= 0 && len != kv_len[p]))) report_status(status, PCP_ERR_RANGE);
    const int32_t full = len / bs, rest = len % bs;
    int32_t fresh = -1, source = -1;
    if (rest > 0) {
        // the child's rank among those that take a page, then the free id of that rank
        int32_t before = 0;
        for (int32_t j = threadIdx.x; j < child; j += kPageThreads) before += tokens_of(j) % bs != 0;
        before = block_sum(before, warp_sums);
        // rounds of kPageThreads chunks: the chunk that holds the free id
        int32_t seen = 0, chunk = -1;
        for (int32_t c0 = 0; c0 < chunks && chunk < 0; c0 += kPageThreads) {
            const int32_t c = c0 + threadIdx.x;
            const int32_t n = c < chunks ? counts[c] : 0;
            const int32_t at = seen + block_before(n, warp_sums);
            if (threadIdx.x == 0) found = -1;
            __syncthreads();
            if (before >= at && before < at + n) found = c;
            __syncthreads();
            chunk = found;
            if (chunk < 0) {
                seen += block_sum(n, warp_sums);
            } else {
                // free ids before the chunk
                seen += block_sum(c < chunk ? n : 0, warp_sums);
            }
        }
        if (chunk >= 0) {
            const int64_t id0 = (int64_t)chunk * kChunk + threadIdx.x * kPer;
            int n = 0;
            const uint32_t live = live_bits(ref, id0, num_blocks, &n);
            const uint32_t free_bits = ~live & (uint32_t)((1ull << n) - 1);
            const int32_t at = seen + block_before(__popc(free_bits), warp_sums);
            if (before >= at && before < at + __popc(free_bits)) {
                uint32_t b = free_bits;
                for (int32_t k = at; k < before; ++k) b &= b - 1;
                found = (int32_t)id0 + __ffs(b) - 1;
            }
            __syncthreads();
            fresh = found;
        }
        const int32_t id = table[(size_t)p * mb + full];
        source = id >= 0 && id < num_blocks && ref[id] > 0 ? id : -1;
        if (threadIdx.x == 0) {
            if (fresh < 0) report_status(status, PCP_ERR_PAGES);
            else if (source < 0) report_status(status, PCP_ERR_RANGE);
            if (fresh >= 0 && source >= 0) ref_out[fresh] = 1;
        }
        if (source < 0) fresh = -1;
    }
    for (int32_t i = threadIdx.x; i < mb; i += kPageThreads) {
        int32_t id = -1;
        if (i < full) {
            id = table[(size_t)p * mb + i];
            if (id >= 0 && id < num_blocks && ref[id] > 0) {
                atomicAdd(ref_out + id, 1);
            } else {
                id = -1;
                report_status(status, PCP_ERR_RANGE);
            }
        } else if (i == full && rest > 0) {
            id = fresh;
        }
        table_out[(size_t)child * mb + i] = id;
    }
    if (fresh >= 0) {
        const int64_t page = (int64_t)bs * vec_per_slot;
        const int32_t n = rest * vec_per_slot;
        for (int32_t i = threadIdx.x; i < n; i += kPageThreads) {
            const uint4 k = kc[source * page + i], v = vc[source * page + i];
            kc[fresh * page + i] = k;
            vc[fresh * page + i] = v;
        }
    }
}

// One block per child.
__global__ void __launch_bounds__(kPageThreads) fork_kernel(ForkArgs f) {
    __shared__ int32_t warp_sums[kPageThreads / 32];
    __shared__ int32_t found;
    grid_wait();
    fork_child(f, blockIdx.x, warp_sums, found);
}

// A whole fork of a few children in one cluster: the counts' copy and the free ids per
// chunk, then the children, dealt to the blocks.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPageThreads) fork_cluster_kernel(ForkArgs f) {
    __shared__ int32_t warp_sums[kPageThreads / 32];
    __shared__ int32_t found;
    for (int32_t c = blockIdx.x; c < f.chunks; c += kCluster) {
        int32_t n = 0;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int64_t i = (int64_t)c * kChunk + e * kPageThreads + threadIdx.x;
            if (i >= f.num_blocks) continue;
            const int32_t r = f.ref[i];
            f.ref_out[i] = r;
            n += r <= 0;
        }
        n = block_sum(n, warp_sums);
        if (threadIdx.x == 0) f.counts[c] = n;
    }
    cluster_sync();
    for (int32_t child = blockIdx.x; child < f.children; child += kCluster) {
        fork_child(f, child, warp_sums, found);
        __syncthreads();  // warp_sums and found are used again
    }
}

// ref_out = ref.
__global__ void __launch_bounds__(kPageThreads)
    copy_counts_kernel(const int32_t* __restrict__ ref, int32_t* __restrict__ ref_out, int64_t num_blocks) {
    grid_launch_dependents();
    const int64_t i = (int64_t)blockIdx.x * kPageThreads + threadIdx.x;
    if (i < num_blocks) ref_out[i] = ref[i];
}

struct ReleaseArgs {
    const int32_t* table;
    int32_t num_reqs, mb;
    const int32_t *first, *last;
    int64_t num_blocks;
    int32_t *table_out, *ref_out;
    int32_t* status;
};

// Entries [first[r], last[r]) of every row give their reference back and become
// -1; entries that are -1 already are passed over. By `threads` threads, this one `tid`.
__device__ __forceinline__ void release_entries(const ReleaseArgs& a, int64_t tid, int64_t threads) {
    const int64_t n = (int64_t)a.num_reqs * a.mb;
    for (int64_t i = tid; i < n; i += threads) {
        const int32_t r = (int32_t)(i / a.mb), col = (int32_t)(i - (int64_t)r * a.mb);
        const int32_t from = __ldg(a.first + r), to = __ldg(a.last + r);
        int32_t id = a.table[i];
        if (from < 0 || to > a.mb) {  // a range outside the row: the row stays as it is
            if (col == 0) report_status(a.status, PCP_ERR_RANGE);
        } else if (col >= from && col < to && id != -1) {
            bool ok = id >= 0 && id < a.num_blocks;
            if (ok && atomicSub(a.ref_out + id, 1) <= 0) {  // nothing left to give back
                atomicAdd(a.ref_out + id, 1);
                ok = false;
            }
            if (!ok) report_status(a.status, PCP_ERR_RANGE);
            id = -1;
        }
        a.table_out[i] = id;
    }
}

__global__ void __launch_bounds__(kPageThreads) release_kernel(ReleaseArgs a) {
    grid_wait();
    release_entries(a, (int64_t)blockIdx.x * kPageThreads + threadIdx.x, (int64_t)gridDim.x * kPageThreads);
}

// The counts' copy and the release in one cluster.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kClusterThreads)
    release_cluster_kernel(ReleaseArgs a, const int32_t* __restrict__ ref) {
    const int64_t tid = (int64_t)blockIdx.x * kClusterThreads + threadIdx.x, threads = kCluster * kClusterThreads;
#pragma unroll 4
    for (int64_t i = tid; i < a.num_blocks; i += threads) a.ref_out[i] = ref[i];
    cluster_sync();
    release_entries(a, tid, threads);
}

// The moves of a compaction. With n live pages, the i-th live id at or above n
// (movers[i]) goes to the i-th free id below n (holes[i]); rank[id] = i for a
// mover. ref_out gets every count but those of the holes. header: n, moves.
__global__ void __launch_bounds__(kPageThreads)
    plan_moves_kernel(const int32_t* __restrict__ ref, int64_t num_blocks, const int32_t* __restrict__ counts,
                      int32_t chunks, int32_t* __restrict__ ref_out, int32_t* __restrict__ holes,
                      int32_t* __restrict__ movers, int32_t* __restrict__ rank, int32_t* header, int32_t* num_live) {
    __shared__ int32_t warp_sums[kPageThreads / 32];
    grid_launch_dependents();
    grid_wait();
    int32_t total = 0, before = 0;
    for (int32_t c = threadIdx.x; c < chunks; c += kPageThreads) {
        const int32_t n = counts[c];
        total += n;
        if (c < (int32_t)blockIdx.x) before += n;
    }
    const int32_t n_live = block_sum(total, warp_sums);
    before = block_sum(before, warp_sums);
    // live ids below n_live: those of the chunks before its own, then within it
    const int32_t edge = n_live / kChunk;
    int32_t below = 0;
    for (int32_t c = threadIdx.x; c < chunks && c < edge; c += kPageThreads) below += counts[c];
    for (int64_t i = (int64_t)edge * kChunk + threadIdx.x; i < n_live; i += kPageThreads) below += ref[i] > 0;
    below = block_sum(below, warp_sums);
    const int64_t id0 = (int64_t)blockIdx.x * kChunk + threadIdx.x * kPer;
    int n = 0;
    const uint32_t live = live_bits(ref, id0, num_blocks, &n);
    int32_t lr = before + block_before(__popc(live), warp_sums);  // live ids before this thread's
    for (int e = 0; e < n; ++e) {
        const int64_t id = id0 + e;
        const bool is_live = (live >> e) & 1;
        if (id < n_live) {
            if (is_live) ref_out[id] = ref[id];
            else holes[id - lr] = (int32_t)id;
        } else {
            ref_out[id] = 0;
            if (is_live) {
                movers[lr - below] = (int32_t)id;
                rank[id] = lr - below;
            }
        }
        lr += is_live;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        header[0] = n_live;
        header[1] = n_live - below;
        if (num_live) *num_live = n_live;
    }
}

// The same in one cluster, counting included: block c has ids [c * per, (c + 1) * per),
// a thread per / kClusterThreads consecutive ones.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kClusterThreads)
    plan_moves_cluster_kernel(const int32_t* __restrict__ ref, int32_t num_blocks, int32_t per_thread, int32_t* counts,
                              int32_t* __restrict__ ref_out, int32_t* __restrict__ holes, int32_t* __restrict__ movers,
                              int32_t* __restrict__ rank, int32_t* header, int32_t* num_live) {
    __shared__ int32_t warp_sums[kClusterThreads / 32];
    grid_launch_dependents();
    const int32_t id0 = ((int32_t)blockIdx.x * kClusterThreads + threadIdx.x) * per_thread;
    const int32_t n = max(0, min(per_thread, num_blocks - id0));
    int32_t r[kClusterPer], mine = 0;
#pragma unroll
    for (int e = 0; e < kClusterPer; ++e) {
        r[e] = e < n ? ref[id0 + e] : 0;
        mine += r[e] > 0;
    }
    const int32_t all = block_sum<kClusterThreads>(mine, warp_sums);
    if (threadIdx.x == 0) counts[blockIdx.x] = all;
    cluster_sync();
    int32_t n_live = 0, before = 0;
#pragma unroll
    for (int c = 0; c < kCluster; ++c) {
        const int32_t k = __ldcg(counts + c);
        n_live += k;
        if (c < (int)blockIdx.x) before += k;
    }
    // live ids below n_live: those of the blocks before its own, then within it
    const int32_t per = kClusterThreads * per_thread, edge = n_live / per;
    int32_t below = 0;
    for (int32_t i = edge * per + threadIdx.x; i < n_live; i += kClusterThreads) below += ref[i] > 0;
    below = block_sum<kClusterThreads>(below, warp_sums);
    for (int c = 0; c < edge; ++c) below += __ldcg(counts + c);
    int32_t lr = before + block_before(mine, warp_sums);  // live ids before this thread's
#pragma unroll
    for (int e = 0; e < kClusterPer; ++e) {
        if (e >= n) break;
        const int32_t id = id0 + e;
        const bool is_live = r[e] > 0;
        if (id < n_live) {
            if (is_live) ref_out[id] = r[e];
            else holes[id - lr] = id;
        } else {
            ref_out[id] = 0;
            if (is_live) {
                movers[lr - below] = id;
                rank[id] = lr - below;
            }
        }
        lr += is_live;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        header[0] = n_live;
        header[1] = n_live - below;
        if (num_live) *num_live = n_live;
    }
}

// The planned moves: K and V of every mover, the holes' counts, and the tables.
__global__ void __launch_bounds__(kCopyThreads)
    move_pages_kernel(uint4* __restrict__ kc, uint4* __restrict__ vc, int32_t page_vec, const int32_t* __restrict__ ref,
                      int64_t num_blocks, const int32_t* __restrict__ holes, const int32_t* __restrict__ movers,
                      const int32_t* __restrict__ rank, const int32_t* __restrict__ header,
                      const int32_t* __restrict__ table, int64_t entries, int32_t* __restrict__ table_out,
                      int32_t* __restrict__ ref_out, int32_t* status) {
    grid_wait();
    const int32_t n_live = header[0], moves = header[1];
    const int64_t tid = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x, step = (int64_t)gridDim.x * kCopyThreads;
    for (int64_t i = tid; i < entries; i += step) {
        const int32_t id = table[i];
        int32_t to = -1;
        if (id >= 0 && id < num_blocks) {
            if (__ldg(ref + id) > 0) to = id < n_live ? id : holes[rank[id]];
        } else if (id != -1) {
            report_status(status, PCP_ERR_RANGE);
        }
        table_out[i] = to;
    }
    for (int64_t i = tid; i < moves; i += step) ref_out[holes[i]] = __ldg(ref + movers[i]);
    // pieces of kCopyThreads x kCopyUnroll vectors of one cache's page, dealt to the blocks
    constexpr int kPiece = kCopyThreads * kCopyUnroll;
    const int32_t pieces = (page_vec + kPiece - 1) / kPiece;
    const int64_t all = (int64_t)moves * pieces * 2;
    for (int64_t p = blockIdx.x; p < all; p += gridDim.x) {
        uint4* cache = (p & 1) ? vc : kc;
        const int64_t m = (p >> 1) / pieces;
        const int32_t at = (int32_t)((p >> 1) - m * pieces) * kPiece + threadIdx.x;
        const uint4* src = cache + (int64_t)movers[m] * page_vec;
        uint4* dst = cache + (int64_t)holes[m] * page_vec;
        uint4 x[kCopyUnroll];
#pragma unroll
        for (int u = 0; u < kCopyUnroll; ++u)
            if (at + u * kCopyThreads < page_vec) x[u] = __ldcs(src + at + u * kCopyThreads);
#pragma unroll
        for (int u = 0; u < kCopyUnroll; ++u)
            if (at + u * kCopyThreads < page_vec) dst[at + u * kCopyThreads] = x[u];
    }
}

int launched(cudaError_t e) {
    if (e != cudaSuccess) {
        set_last_cuda_error(e);
        return PCP_ERR_CUDA;
    }
    return PCP_OK;
}

// The arguments that fork and compaction share.
int check_pages(const void* kc, const void* vc, int64_t num_blocks, int32_t bs, int32_t slot_bytes, int32_t num_reqs,
                int32_t mb) {
    if (num_blocks < 0 || num_blocks > INT32_MAX || bs < 1 || slot_bytes < 1 || num_reqs < 0 || mb < 0)
        return PCP_ERR_ARG;
    if ((int64_t)mb * bs > INT32_MAX || (int64_t)bs * slot_bytes > INT32_MAX) return PCP_ERR_ARG;
    if (slot_bytes % 16 != 0) return PCP_ERR_UNSUPPORTED;
    if (num_blocks > 0 && (!kc || !vc)) return PCP_ERR_ARG;
    if (!aligned16(kc) || !aligned16(vc)) return PCP_ERR_ALIGN;
    return PCP_OK;
}

}  // namespace

}  // namespace pcp

using namespace pcp;

extern "C" size_t pcp_kv_pages_workspace_size(int64_t num_blocks) {
    if (num_blocks < 0 || num_blocks > INT32_MAX) return 0;
    return pages_layout(num_blocks).total;
}

extern "C" int pcp_kv_fork(void* key_cache, void* value_cache, int64_t num_blocks, int32_t block_size,
                           int32_t slot_bytes, const int32_t* block_table, int32_t num_reqs,
                           int32_t max_blocks_per_req, const int32_t* kv_len, const int32_t* parent,
                           int32_t num_children, const int32_t* ref_count, int32_t* block_table_out,
                           int32_t* ref_count_out, void* workspace, size_t workspace_bytes, int32_t* status,
                           pcp_stream_t stream) {
    const int rc = check_pages(key_cache, value_cache, num_blocks, block_size, slot_bytes, num_reqs,
                               max_blocks_per_req);
    if (rc != PCP_OK) return rc;
    if (num_children < 0) return PCP_ERR_ARG;
    if (num_blocks == 0) return num_children == 0 ? PCP_OK : PCP_ERR_ARG;
    if (!ref_count || !ref_count_out || !workspace ||
        (num_children > 0 && (!parent || (num_reqs > 0 && !kv_len) ||
                              (max_blocks_per_req > 0 && (!block_table_out || (num_reqs > 0 && !block_table))))))
        return PCP_ERR_ARG;
    if (!aligned4(block_table) || !aligned4(kv_len) || !aligned4(parent) || !aligned4(ref_count) ||
        !aligned4(block_table_out) || !aligned4(ref_count_out) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return PCP_ERR_ALIGN;
    const PagesLayout w = pages_layout(num_blocks);
    if (workspace_bytes < w.total) return PCP_ERR_WORKSPACE;
    const size_t cache = (size_t)num_blocks * block_size * slot_bytes, ref = (size_t)num_blocks * 4;
    const Span outs[5] = {{key_cache, cache},
                          {value_cache, cache},
                          {block_table_out, (size_t)num_children * max_blocks_per_req * 4},
                          {ref_count_out, ref},
                          {workspace, w.total}};
    const Span ins[4] = {{block_table, (size_t)num_reqs * max_blocks_per_req * 4},
                         {kv_len, (size_t)num_reqs * 4},
                         {parent, (size_t)num_children * 4},
                         {ref_count, ref}};
    for (int i = 0; i < 5; ++i)
        if (overlaps_any(outs[i], ins, 4) || overlaps_any(outs[i], outs + i + 1, 4 - i)) return PCP_ERR_ARG;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int32_t* counts = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + w.counts);
    const ForkArgs f{static_cast<uint4*>(key_cache), static_cast<uint4*>(value_cache), num_blocks, block_size,
                     slot_bytes / 16, block_table, num_reqs, max_blocks_per_req, kv_len, parent, num_children, ref_count,
                     block_table_out, ref_count_out, counts, w.chunks, status};
    if (num_children <= kClusterChildren && num_blocks <= kClusterIds) {
        fork_cluster_kernel<<<kCluster, kPageThreads, 0, s>>>(f);
        return launched(cudaGetLastError());
    }
    count_kernel<true><<<w.chunks, kPageThreads, 0, s>>>(ref_count, ref_count_out, num_blocks, counts);
    const int e = launched(cudaGetLastError());
    if (e != PCP_OK || num_children == 0) return e;
    return launched(launch_chained(fork_kernel, dim3(num_children), dim3(kPageThreads), 0, s, f));
}

extern "C" int pcp_kv_release(const int32_t* block_table, int32_t num_reqs, int32_t max_blocks_per_req,
                              const int32_t* first_page, const int32_t* last_page, const int32_t* ref_count,
                              int64_t num_blocks, int32_t* block_table_out, int32_t* ref_count_out, int32_t* status,
                              pcp_stream_t stream) {
    if (num_reqs < 0 || max_blocks_per_req < 0 || num_blocks < 0 || num_blocks > INT32_MAX) return PCP_ERR_ARG;
    const int64_t entries = (int64_t)num_reqs * max_blocks_per_req;
    if ((num_blocks > 0 && (!ref_count || !ref_count_out)) ||
        (entries > 0 && (!block_table || !block_table_out || !first_page || !last_page)))
        return PCP_ERR_ARG;
    if (!aligned4(block_table) || !aligned4(first_page) || !aligned4(last_page) || !aligned4(ref_count) ||
        !aligned4(block_table_out) || !aligned4(ref_count_out))
        return PCP_ERR_ALIGN;
    const Span table{block_table, (size_t)entries * 4}, table_out{block_table_out, (size_t)entries * 4};
    const Span ref{ref_count, (size_t)num_blocks * 4}, ref_out{ref_count_out, (size_t)num_blocks * 4};
    const Span ranges[2] = {{first_page, (size_t)num_reqs * 4}, {last_page, (size_t)num_reqs * 4}};
    // each output is its input's buffer or clear of it, and clear of everything else
    if ((block_table != block_table_out && overlap(table, table_out)) || (ref_count != ref_count_out && overlap(ref, ref_out)) ||
        overlap(table_out, ref_out) || overlap(table_out, ref) || overlap(ref_out, table) ||
        overlaps_any(table_out, ranges, 2) || overlaps_any(ref_out, ranges, 2))
        return PCP_ERR_ARG;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const ReleaseArgs a{block_table, num_reqs, max_blocks_per_req, first_page, last_page, num_blocks, block_table_out,
                        ref_count_out, status};
    const bool copy = ref_count != ref_count_out && num_blocks > 0;
    if (copy && num_blocks <= kClusterIds && entries <= kClusterEntries) {
        release_cluster_kernel<<<kCluster, kClusterThreads, 0, s>>>(a, ref_count);
        return launched(cudaGetLastError());
    }
    if (copy) {
        copy_counts_kernel<<<(unsigned)((num_blocks + kPageThreads - 1) / kPageThreads), kPageThreads, 0, s>>>(
            ref_count, ref_count_out, num_blocks);
        const int e = launched(cudaGetLastError());
        if (e != PCP_OK) return e;
    }
    if (entries == 0) return PCP_OK;
    int64_t blocks = (entries + kPageThreads - 1) / kPageThreads;
    const int64_t cap = (int64_t)num_sms() * 8;
    if (blocks > cap) blocks = cap;
    if (!copy) {  // nothing of this call to be chained behind
        release_kernel<<<(unsigned)blocks, kPageThreads, 0, s>>>(a);
        return launched(cudaGetLastError());
    }
    return launched(launch_chained(release_kernel, dim3((unsigned)blocks), dim3(kPageThreads), 0, s, a));
}

extern "C" int pcp_kv_compact(void* key_cache, void* value_cache, int64_t num_blocks, int32_t block_size,
                              int32_t slot_bytes, const int32_t* block_table, int32_t num_reqs,
                              int32_t max_blocks_per_req, const int32_t* ref_count, int32_t* block_table_out,
                              int32_t* ref_count_out, int32_t* num_live, void* workspace, size_t workspace_bytes,
                              int32_t* status, pcp_stream_t stream) {
    const int rc = check_pages(key_cache, value_cache, num_blocks, block_size, slot_bytes, num_reqs,
                               max_blocks_per_req);
    if (rc != PCP_OK) return rc;
    const int64_t entries = (int64_t)num_reqs * max_blocks_per_req;
    if (num_blocks == 0) return PCP_ERR_ARG;
    if (!ref_count || !ref_count_out || !workspace || (entries > 0 && (!block_table || !block_table_out)))
        return PCP_ERR_ARG;
    if (!aligned4(block_table) || !aligned4(ref_count) || !aligned4(block_table_out) || !aligned4(ref_count_out) ||
        !aligned4(num_live) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return PCP_ERR_ALIGN;
    const PagesLayout w = pages_layout(num_blocks);
    if (workspace_bytes < w.total) return PCP_ERR_WORKSPACE;
    const size_t cache = (size_t)num_blocks * block_size * slot_bytes, ref = (size_t)num_blocks * 4;
    const Span outs[6] = {{key_cache, cache},
                          {value_cache, cache},
                          {block_table_out, (size_t)entries * 4},
                          {ref_count_out, ref},
                          {num_live, num_live ? size_t(4) : 0},
                          {workspace, w.total}};
    const Span ins[2] = {{block_table, (size_t)entries * 4}, {ref_count, ref}};
    for (int i = 0; i < 6; ++i)
        if (overlaps_any(outs[i], ins, 2) || overlaps_any(outs[i], outs + i + 1, 5 - i)) return PCP_ERR_ARG;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    auto ints = [&](size_t at) { return reinterpret_cast<int32_t*>(ws + at); };
    int e;
    if (num_blocks <= kClusterIds) {
        const int32_t per = (int32_t)((num_blocks + kCluster * kClusterThreads - 1) / (kCluster * kClusterThreads));
        plan_moves_cluster_kernel<<<kCluster, kClusterThreads, 0, s>>>(
            ref_count, (int32_t)num_blocks, per, ints(w.header) + 8, ref_count_out, ints(w.holes), ints(w.movers),
            ints(w.rank), ints(w.header), num_live);
        e = launched(cudaGetLastError());
    } else {
        count_kernel<false><<<w.chunks, kPageThreads, 0, s>>>(ref_count, nullptr, num_blocks, ints(w.counts));
        e = launched(cudaGetLastError());
        if (e != PCP_OK) return e;
        e = launched(launch_chained(plan_moves_kernel, dim3(w.chunks), dim3(kPageThreads), 0, s, ref_count, num_blocks,
                                    ints(w.counts), w.chunks, ref_count_out, ints(w.holes), ints(w.movers),
                                    ints(w.rank), ints(w.header), num_live));
    }
    if (e != PCP_OK) return e;
    return launched(launch_chained(move_pages_kernel, dim3(num_sms() * 4), dim3(kCopyThreads), 0, s,
                                   static_cast<uint4*>(key_cache), static_cast<uint4*>(value_cache),
                                   block_size * (slot_bytes / 16), ref_count, num_blocks, ints(w.holes),
                                   ints(w.movers), ints(w.rank), ints(w.header), block_table, entries,
                                   block_table_out, ref_count_out, status));
}
