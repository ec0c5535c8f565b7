// One-token rows of the window and shared-prefix calls on the 5th-generation tensor
// cores (head_dim 128): each row attends the keys of its own walk (KeyRange: sinks
// and window, or what follows its shared prefix).
//
// The products are those of decode_tc_kernel (S^T = K Q^T with the keys along M,
// O^T = V^T P^T, P as hi + lo); what differs is how the work is spread. These rows
// have few keys (a window, a suffix), often one or two 128-key tiles per item, and
// an item's start and end (its first tile's way through the pipeline, the sums over
// the warps, the result) cost more than a tile. decode_tc_kernel shares an item's
// tiles between its two softmax warpgroups and joins them at the item's end, where
// both wait; here each warpgroup has an item of its own:
//  * a CTA takes its items two at a time (items 2q and 2q + 1 of its share), one per
//    warpgroup, their tiles interleaved in one stream (tile j of the first, tile j of
//    the second, ...): the rings, the MMA issuers and the q warps follow that stream,
//    and one item's start and end run under the other's tiles. Measured against the
//    shared items: 64 rows of 16 to 512 keys on 61 SMs 39 -> 31 us, 128 rows of 4132
//    slots over an e4m3 cache 219 -> 214 us;
//  * an item has one partial, or is the row's result itself where the call's rows
//    are one split each (a.direct);
//  * e4m3 cache: PV takes the V codes as they are too (A MN-major, 32 keys per MMA):
//    P goes in as three e4m3 terms, p 2^8, then the remainder 2^12, then its remainder
//    2^16 (each term keeps 4 significant bits, so a remainder is at most 2^-4 of what it
//    remains of and stays below e4m3's 448), in columns of their own, whose O^T the
//    softmax joins with the powers of two taken back: 12 significant bits of p, and
//    2^-26 of the row's largest weight where a term is subnormal. No V is widened, and
//    the rings hold six 16 KB tiles of K and of V. Measured against V widened to f16
//    by converter warps: 128 rows of 4132 slots 214 -> 182 us (5.7 TB/s);
//  * each warpgroup has its own S, P and O buffer; Q^T has two buffers per
//    warpgroup (one with 16 heads, for lack of shared memory);
//  * the producers look one tile ahead: a tile's pages, and behind an item's last
//    tile the next items' records, are read before the wait for the current stage.
// Launched behind the scheduler (launch_chained), on header[2] of the SMs. A call of
// a few one-token rows whose items all fit the SMs at once (a.inline_items) has no
// scheduler: one warp of each CTA reads the rows (kInlineRows at most) and finds
// the CTA's two items itself. Measured, 4 rows with a window of 1024: 18.5 -> 16.4 us.
// Nor has it a merge where a cluster can take each row and kv head (a.cluster): its
// blocks have two splits each and join them through each other's shared memory; the
// call is this one kernel. 4 rows 16.4 -> 14.4 us, 1 row 14.4 -> 10.5, 8 rows with a
// window of 16384 95 -> 85 us; 8 rows behind 1008 shared keys 25.3 -> 16.4 (see decode_cluster).
//
// What bounds it: HBM with a bf16 cache where the rows fill the SMs (56 rows of 1060
// slots: 242 MB in 46 us, 5.3 TB/s; 128 of 4132 over an e4m3 cache: 1.04 GB in 182 us,
// 5.7 TB/s, 84 % of a copy's), the latency of one pair of items in small calls.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "decode_tc_parts.cuh"
#include "pcp_device.cuh"
#include "pcp_internal.h"

namespace pcp {

namespace {

template <bool F8, int GP>
struct PairCfg {
    static constexpr int kNS = 16;                     // S^T columns: the q heads, or their e4m3 terms
    static constexpr int kGS = GP <= 8 ? 8 : 16;       // head stride of the per-head arrays
    // O^T columns, P^T rows: P's hi parts, then the remainders (bf16: two terms; e4m3: three)
    static constexpr int kTS = F8 ? (GP <= 4 ? 4 : 8) : kGS;  // columns per term
    static constexpr int kNO = F8 ? (GP <= 4 ? 16 : 32) : 2 * kGS;
    static constexpr int kKS = F8 ? 6 : 3;             // K tiles in flight
    static constexpr int kVS = F8 ? 6 : 3;             // V tiles in flight
    static constexpr int kQB = GP <= 8 ? 2 : 1;        // Q^T buffers per warpgroup
    static constexpr int kHalfBytes = kKeys * 128;
    static constexpr int kTileBytes = F8 ? kHalfBytes : 2 * kHalfBytes;  // 128 keys x 128 dims
    static constexpr int kRowsBytes = kN * 128;
    static constexpr int kQBytes = 2 * kRowsBytes;
    static constexpr int kQCBytes = F8 ? kNS * 128 : 0;
    static constexpr int kPBytes = (F8 ? 1 : 2) * kNO * 128;
    static constexpr int kK = 0;
    static constexpr int kV = kKS * kTileBytes;
    static constexpr int kQ = kV + kVS * kTileBytes;   // [warpgroup + 2 x buffer]
    static constexpr int kQC = kQ + 2 * kQB * kQBytes;
    static constexpr int kP = kQC + 2 * kQB * kQCBytes;
    static constexpr int kRed = kP + 2 * kPBytes;      // float [2 wg][2 tile parities][4 warps][head]: maxima
    static constexpr int kSum = kRed + 2 * 2 * 4 * kGS * 4;  // float [2 wg][2 item parities][4 warps][head]
    // FP8 q scales, float [warpgroup + 2 x (pair mod 4)][head]: those of pair q + 4 are written
    // once its q has landed, which needs S of pair q + 2's last tile (kQB = 2), which
    // needs the softmax in pair q + 1, past its reading of pair q's
    static constexpr int kQs = kSum + 2 * 2 * 4 * kGS * 4;
    static constexpr int kBar = kQs + 8 * kGS * 4;
    static constexpr int kNumBars = 2 * kKS + 2 * kVS + 3 * 2 * kQB + 8 + 4 * 2;
    static constexpr int kThreads = 32 * (F8 ? 16 : 12);  // e4m3: four warps turn q into its terms
    static constexpr int kMisc = kBar + kNumBars * 8;  // TMEM address, abort flag, item count
    static constexpr int kOwn = kMisc + 16;            // PairItem [2]: a.inline_items
    static constexpr int kSmem = kOwn + 2 * 44 + 1024;  // + alignment slack
    static constexpr uint32_t kTmemS = 0, kTmemO = 2 * kNS;
    static constexpr uint32_t kTmemCols = 2 * kNS + 2 * kNO <= 64 ? 64 : 128;
    static constexpr uint32_t kIdescS = F8 ? idesc_e4m3(128, kNS) : idesc_bf16(128, kN, false, false);
    static constexpr uint32_t kIdescO = F8 ? idesc_e4m3(128, kNO, true) : idesc_bf16(128, kNO, true, false);
};
static_assert(PairCfg<true, 4>::kSmem <= 232448 && PairCfg<true, 8>::kSmem <= 232448 &&
                  PairCfg<false, 8>::kSmem <= 232448 && PairCfg<false, 16>::kSmem <= 232448, "shared memory");
static_assert(PairCfg<true, 4>::kQC % 1024 == 0 && PairCfg<true, 4>::kP % 1024 == 0 &&
                  PairCfg<true, 8>::kP % 1024 == 0 && PairCfg<false, 8>::kP % 1024 == 0 &&
                  PairCfg<false, 16>::kP % 1024 == 0, "1024-byte swizzle atoms");

// An item: a split of one row for one kv head; nt 0: none.
struct PairItem {
    int32_t row, req, q_start, hk, lo, hi, nt;  // slots [lo, hi) of the row's walk, in nt tiles
    int32_t sinks, gap_end, shift;
    int32_t preq;  // request whose table names the pages of the sinks (a.cluster: or of the shared prefix)
    // whether slot v holds a key that the row sees
    __device__ __forceinline__ bool live(int32_t v) const { return v < sinks || v >= gap_end; }
};

__device__ __forceinline__ PairItem pair_item(const PrefillArgs& a, int32_t p, int32_t total) {
    PairItem it{};
    if (p < 0 || p >= total) return it;
    const int32_t n = p / a.hkv;
    const int4* src = reinterpret_cast<const int4*>(a.dec_units + n);
    const int4 x = src[0], y = src[1];
    it.row = x.x;
    it.req = x.y;
    it.q_start = x.z;
    it.hk = p - n * a.hkv;
    it.lo = x.w;
    it.hi = y.x;
    it.sinks = y.y;
    it.gap_end = y.z;
    it.shift = y.w;
    it.preq = it.req;
    it.nt = (it.hi - it.lo + kKeys - 1) / kKeys;
    return it;
}

static_assert(sizeof(PairItem) == 44, "two of them fit at PairCfg::kOwn");

// e4m3 cache: the V descales of an item's own keys and of those it walks as sinks (a shared
// prefix's are its request's), as a factor at most 1 on P for each and one on the result.
struct VScale {
    float all, own, pre;
};
__device__ __forceinline__ VScale v_scale(const PrefillArgs& a, const PairItem& it) {
    const float own = __ldg(a.v_descale + (size_t)it.req * a.hkv + it.hk);
    const float pre = it.preq == it.req ? own : __ldg(a.v_descale + (size_t)it.preq * a.hkv + it.hk);
    if (own == pre) return {own, 1.f, 1.f};
    const float all = fmaxf(fabsf(own), fabsf(pre));
    return {all, own / all, pre / all};
}

// a.inline_items: one warp's work of finding the items `p0` and `p1` (-1: none) among
// all rows, splits and kv heads (row by row, split by split, head by head); returns
// the item count. CTA 0 also reports bad rows and writes the merge records.
constexpr int kInlineRows = 64;
constexpr int kMaxCluster = 8;  // blocks of a cluster at most (a.cluster)
constexpr int kPrefixKeys = 1024;  // keys of a split at most where rows read a shared prefix each
__device__ __forceinline__ int32_t inline_items(const PrefillArgs& a, int32_t p0, int32_t p1, PairItem* own,
                                                int lane) {
    constexpr int kPer = kInlineRows / 32;
    const int64_t max_kv = (int64_t)a.max_blocks * a.block_size;
    pcp_row_t row[kPer];
    KeyRange kr[kPer];
    int32_t splits[kPer], before[kPer], sum = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int32_t ri = lane * kPer + k;
        row[k] = ri < a.num_rows ? a.rows[ri] : pcp_row_t{};
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int32_t ri = lane * kPer + k;
        const bool ok = ri < a.num_rows && row_in_range(row[k], a.num_reqs, a.total_q, max_kv) && row[k].q_len == 1;
        if (!ok) row[k].kv_end = 0;
        kr[k] = key_range(a, row[k], 0);
        splits[k] = ok ? (kr[k].len + a.chunk - 1) / a.chunk : 0;
        sum += splits[k];
        if (blockIdx.x == 0 && ri < a.num_rows) {
            if (!ok) report_status(a.status, PCP_ERR_RANGE);
            a.merge[ri] = MergeTask{ok ? ri : -1, row[k].q_start, splits[k], 0};
        }
    }
    int32_t at = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t x = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += x;
    }
    const int32_t total = __shfl_sync(0xffffffffu, at, 31) * a.hkv;
    at -= sum;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        before[k] = at;
        at += splits[k];
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const int32_t p = w ? p1 : p0;
        if (p < 0 || p >= total) {
            if (lane == 0) own[w] = PairItem{};
            continue;
        }
        const int32_t n = p / a.hkv;
#pragma unroll
        for (int k = 0; k < kPer; ++k)
            if (n >= before[k] && n < before[k] + splits[k]) {
                PairItem it;
                it.row = lane * kPer + k;
                it.req = it.preq = row[k].req;
                it.q_start = row[k].q_start;
                it.hk = p - n * a.hkv;
                it.lo = (n - before[k]) * a.chunk;
                it.hi = min(kr[k].len, it.lo + a.chunk);
                it.nt = (it.hi - it.lo + kKeys - 1) / kKeys;
                it.sinks = kr[k].sinks;
                it.gap_end = kr[k].lo - kr[k].shift;
                it.shift = kr[k].shift;
                own[w] = it;
            }
    }
    return total;
}

// a.cluster: one warp's work of finding the block's two items, splits 2 x rank and 2 x
// rank + 1 of the cluster's row and kv head; returns how many of them there are, and in
// *splits those of the cluster. The splits are as even as whole tiles allow. A shared
// prefix is walked as sinks are, its pages those of the group's request; a row begins at
// or past its prefix, so its own pages follow, the first one again where the prefix ends
// inside a page.
constexpr int kClusterGroups = 16;  // prefix groups at most (every block checks them)
__device__ __forceinline__ int32_t cluster_items(const PrefillArgs& a, PairItem* own, int32_t* splits, int lane) {
    const int32_t unit = (int32_t)blockIdx.x / a.cluster, rank = (int32_t)blockIdx.x - unit * a.cluster;
    const int32_t ri = unit / a.hkv, ng = a.num_prefixes;
    const int64_t max_kv = (int64_t)a.max_blocks * a.block_size;
    pcp_prefix_t p{};
    if (lane < ng) p = a.prefixes[lane];
    pcp_row_t row = a.rows[ri];
    bool ok = row_in_range(row, a.num_reqs, a.total_q, max_kv) && row.q_len == 1;
    int32_t prefix = 0, preq = row.req;
    if (ng > 0) {
        // the group of this lane: fields in range, and its tokens after those of every earlier group
        bool good = p.q_start >= 0 && p.q_len >= 1 && (int64_t)p.q_start + p.q_len <= a.total_q && p.req >= 0 &&
                    p.req < a.num_reqs && p.prefix_len >= 1 && p.prefix_len <= max_kv;
        const int64_t p1 = (int64_t)p.q_start + p.q_len;
        for (int e = 0; e + 1 < ng; ++e) {
            const int64_t end = __shfl_sync(0xffffffffu, p1, e);
            if (lane > e) good = good && p.q_start >= end;
        }
        if (blockIdx.x == 0 && lane < ng && !good) report_status(a.status, PCP_ERR_RANGE);
        // the row's group, which has to be good and to end where the row begins or before
        const bool mine = lane < ng && row.q_start >= p.q_start && row.q_start < p1;
        ok = ok && __all_sync(0xffffffffu, !mine || (good && row.kv_end - 1 >= p.prefix_len));
        const uint32_t which = __ballot_sync(0xffffffffu, mine);
        const int src = which ? __ffs(which) - 1 : 0;
        const int32_t len = __shfl_sync(0xffffffffu, p.prefix_len, src), req = __shfl_sync(0xffffffffu, p.req, src);
        if (which && ok) {
            prefix = len;
            preq = req;
        }
    }
    if (!ok) row.kv_end = 0;
    KeyRange kr = key_range(a, row, 0);
    if (prefix > 0) {
        const int32_t bs = a.block_size;
        kr.lo = kr.sinks = prefix;
        kr.shift = prefix / bs * bs - (prefix + bs - 1) / bs * bs;
        kr.len = row.kv_end - kr.shift;
    }
    PairItem it{};
    it.row = ri;
    it.req = row.req;
    it.preq = preq;
    it.q_start = row.q_start;
    it.hk = unit - ri * a.hkv;
    it.sinks = kr.sinks;
    it.gap_end = kr.lo - kr.shift;
    it.shift = kr.shift;
    if (!ok && rank == 0 && it.hk == 0 && lane == 0) report_status(a.status, PCP_ERR_RANGE);
    const int32_t tiles = (kr.len + kKeys - 1) / kKeys, chunk = max(1, (tiles + 2 * a.cluster - 1) / (2 * a.cluster)) * kKeys;
    int32_t n = 0;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        it.lo = (2 * rank + w) * chunk;
        it.hi = min(kr.len, it.lo + chunk);
        it.nt = it.hi > it.lo ? (it.hi - it.lo + kKeys - 1) / kKeys : 0;
        n += it.nt > 0;
        if (lane == 0) own[w] = it;
    }
    *splits = (kr.len + chunk - 1) / chunk;
    return n;
}

template <bool F8, int GP>
__global__ void __launch_bounds__(PairCfg<F8, GP>::kThreads, 1)
    decode_pair_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, PrefillArgs a, float* __restrict__ dec_out,
                       float* __restrict__ dec_lse, int max_splits, int q_rows) {
    using C = PairCfg<F8, GP>;
    constexpr int kKS = C::kKS, kVS = C::kVS, kNS = C::kNS, kGS = C::kGS, kNO = C::kNO, kQB = C::kQB, kTS = C::kTS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar0 = sbase + C::kBar;
    // stage barriers: K tile landed, K stage free (its S is done); V the same (its PV)
    auto k_full = [&](int s) { return bar0 + 8 * s; };
    auto k_empty = [&](int s) { return bar0 + 8 * (kKS + s); };
    const uint32_t bv = bar0 + 8 * 2 * kKS;
    auto v_full = [&](int s) { return bv + 8 * s; };
    auto v_empty = [&](int s) { return bv + 8 * (kVS + s); };
    // per Q^T buffer: ready / bf16 landed (FP8) / free; FP8: q scales of a slot written
    const uint32_t bq = bv + 8 * 2 * kVS;
    auto q_full = [&](int b) { return bq + 8 * b; };
    auto qc_full = [&](int b) { return bq + 8 * (2 * kQB + b); };
    auto q_empty = [&](int b) { return bq + 8 * (4 * kQB + b); };
    auto q_ready = [&](int n) { return bq + 8 * (6 * kQB + n); };
    // per warpgroup: S^T, P^T, O^T written, O^T taken
    const uint32_t bx = bq + 8 * (6 * kQB + 8);
    auto s_full = [&](int w) { return bx + 8 * w; };
    auto p_full = [&](int w) { return bx + 16 + 8 * w; };
    auto o_full = [&](int w) { return bx + 32 + 8 * w; };
    auto o_free = [&](int w) { return bx + 48 + 8 * w; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMisc + 4);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int G = a.hq / a.hkv;
    const int32_t bs = a.block_size;
    if (threadIdx.x == 0) {
        const uint32_t filled = F8 ? 4 : 1;  // FP8: each warp of the converter set arrives
        for (int s = 0; s < kKS; ++s) {
            mbar_init(k_full(s), 1);
            mbar_init(k_empty(s), 1);
        }
        for (int s = 0; s < kVS; ++s) {
            mbar_init(v_full(s), 1);
            mbar_init(v_empty(s), 1);
        }
        for (int b = 0; b < 2 * kQB; ++b) {
            mbar_init(q_full(b), filled);
            mbar_init(qc_full(b), 1);
            mbar_init(q_empty(b), 1);
        }
        for (int n = 0; n < 8; ++n) mbar_init(q_ready(n), 4);
        for (int w = 0; w < 2; ++w) {
            mbar_init(s_full(w), 1);
            mbar_init(p_full(w), 4);  // the warpgroup's four warps
            mbar_init(o_full(w), 1);
            mbar_init(o_free(w), 4);
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
        tmem_relinquish();
    }
    if (warp == kProdWarp && lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    PairItem* own = reinterpret_cast<PairItem*>(smem + C::kOwn);
    int32_t* own_total = reinterpret_cast<int32_t*>(smem + C::kMisc + 8);
    int32_t* row_splits = own_total + 1;  // a.cluster: splits of the cluster's row
    if (a.inline_items) {
        grid_launch_dependents();
        if (warp == 0) {
            int32_t n, splits = 0;
            if (a.cluster) n = cluster_items(a, own, &splits, lane);
            else n = inline_items(a, (int32_t)blockIdx.x, 2 * a.num_sms - 1 - (int32_t)blockIdx.x, own, lane);
            if (lane == 0) {
                *own_total = n;
                *row_splits = splits;
            }
        }
        __syncthreads();
    } else {
        // the scheduler's lists are read from here on
        grid_wait();
        grid_launch_dependents();
    }
    // CTAs that take items: as many as the scheduler gave the decode rows. Items in
    // snake order (forward on even rounds, backward on odd ones) over the list, longest
    // first; rounds 2q and 2q + 1 are pair q.
    const int32_t step = a.inline_items ? a.num_sms : a.num_units[2];
    const int32_t total = a.inline_items ? *own_total : (int32_t)blockIdx.x < step ? a.num_units[1] : 0;
    // (A CTA without items gets `total` in every round: the snake's backward rounds
    // would be negative for it.)
    auto item_of_round = [&](int32_t rd) -> int32_t {
        if (a.cluster) return rd;  // `total` items, of rounds 0 and 1
        if ((int32_t)blockIdx.x >= step) return total;
        return rd * step + ((rd & 1) ? step - 1 - (int32_t)blockIdx.x : (int32_t)blockIdx.x);
    };
    auto item_at = [&](int32_t rd) -> PairItem {
        if (a.inline_items) return rd < 2 ? own[rd] : PairItem{};
        return pair_item(a, item_of_round(rd), total);
    };
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // Q^T buffer of pair q's item w, and the parity of its use
    auto q_buf = [&](int32_t q, int w) { return w + 2 * (kQB == 2 ? (q & 1) : 0); };
    auto q_use = [&](int32_t q) -> uint32_t { return (kQB == 2 ? q >> 1 : q) & 1; };
    auto qs_slot = [&](int32_t q, int w) { return w + 2 * (q & 3); };  // FP8: of its q scales

    if (warp == kProdWarp || warp == kProdWarp + 1) {
        // ---------------------------------------------------------------- producers
        // Warp 8 loads the K tiles (and each item's Q^T before its first), warp 9 the V
        // tiles. Lane p owns page p of every tile.
        const bool is_k = warp == kProdWarp;
        const CUtensorMap* tm = is_k ? &tm_k : &tm_v;
        const int nst = is_k ? kKS : kVS;
        const int32_t oob = (int32_t)(a.num_blocks * bs);  // a row past the cache: zero fill
        const uint32_t q_bytes = 2u * (uint32_t)q_rows * 128u;
        auto full_of = [&](int st) { return is_k ? k_full(st) : v_full(st); };
        // cursor over the stream: tile j of item w of pair q
        PairItem i0 = item_at(0), i1 = item_at(1);
        int32_t q = 0, j = 0;
        int w = 0;
        auto cur = [&]() -> const PairItem& { return w ? i1 : i0; };
        // this lane's page id of the cursor's tile, read ahead and looked at only when the tile
        // is loaded (a test of it here would wait for it)
        auto page_id = [&]() -> int32_t {
            const PairItem& it = cur();
            const int32_t v = it.lo + j * kKeys + lane * bs;
            const int32_t pg = (v >= it.sinks ? v + it.shift : v) / bs;  // a page begun by sinks holds them
            if (lane * bs >= kKeys || v >= it.hi || pg >= a.max_blocks) return -1;
            return __ldg(a.block_table + (size_t)(v >= it.sinks ? it.req : it.preq) * a.max_blocks + pg);
        };
        bool ok = true;
        uint32_t gt = 0, uses[2] = {0, 0};  // tiles; items with a Q^T load per warpgroup
        int32_t id = i0.nt > 0 ? page_id() : -1;
        while (cur().nt > 0) {
            const bool first = j == 0;
            const int32_t nvalid = min(kKeys, cur().hi - cur().lo - j * kKeys), hk = cur().hk, q_tok = cur().q_start;
            const int np = (nvalid + bs - 1) / bs, qb = q_buf(q, w);
            const uint32_t qp = q_use(q) ^ 1;
            // on to the next tile, its pages read before the waits below
            const bool other = w == 0 ? j < i1.nt : j + 1 < i0.nt;  // the other item has the next tile
            if (other) {
                j += w;
                w ^= 1;
            } else if (j + 1 < cur().nt) {
                ++j;
            } else {
                ++q;
                i0 = item_at(2 * q);
                i1 = item_at(2 * q + 1);
                w = 0;
                j = 0;
            }
            const int32_t id_next = cur().nt > 0 ? page_id() : -1;
            if (is_k && first) {
                if (!(ok = mbar_wait_warp(q_empty(qb), qp, abort_flag))) break;
                if (lane == 0) {
                    const uint32_t qbar = F8 ? qc_full(qb) : q_full(qb);
                    mbar_arrive_expect_tx(qbar, q_bytes);
                    for (int h = 0; h < 2; ++h)
                        tma_load_3d(sbase + C::kQ + qb * C::kQBytes + h * C::kRowsBytes, &tm_q, qbar, h * 64, hk * G,
                                    q_tok);
                }
                ++uses[qb & 1];
            }
            const int st = gt % nst;
            if (!(ok = mbar_wait_warp(is_k ? k_empty(st) : v_empty(st), ((gt / nst) & 1) ^ 1, abort_flag))) break;
            const uint32_t fb = full_of(st);
            if (lane == 0) mbar_arrive_expect_tx(fb, (uint32_t)(np * bs) * (F8 ? kD : 2 * kD));
            __syncwarp();
            if (lane < np) {
                // a bad id maps to a row past the cache (zero filled) and is reported
                const bool good = id >= 0 && id < a.num_blocks;
                if (!good && is_k) report_status(a.status, PCP_ERR_RANGE);
                const int32_t y = good ? id * bs : oob;
                const uint32_t dst = sbase + (is_k ? C::kK : C::kV) + st * C::kTileBytes;
                if constexpr (F8) {  // the codes, 128-byte swizzled, as the e4m3 operands
                    tma_load_3d(dst + lane * bs * kD, tm, fb, 0, hk, y);
                } else {
                    for (int h = 0; h < 2; ++h)
                        tma_load_3d(dst + h * C::kHalfBytes + lane * bs * 128, tm, fb, h * 64, hk, y);
                }
            }
            ++gt;
            id = id_next;
        }
        if (!ok && lane == 0) {
            report_status(a.status, PCP_ERR_TIMEOUT);
            // wait (bounded, whatever the abort flag says) for the copies already
            // issued, so that none lands after the CTA has gone
            int no_abort = 0;
            for (uint32_t g = gt > (uint32_t)nst ? gt - nst : 0; g < gt; ++g)
                mbar_wait(full_of(g % nst), (g / nst) & 1, &no_abort, 100000000ull);
            if (is_k)
                for (int b = 0; b < 2 * kQB; ++b) {
                    // the last use of buffer b: uses of its warpgroup, every kQB-th of them
                    const uint32_t n = uses[b & 1], first_use = b >> 1;
                    if (n > first_use)
                        mbar_wait(F8 ? qc_full(b) : q_full(b), ((n - 1 - first_use) / kQB) & 1, &no_abort, 100000000ull);
                }
        }
    } else if (warp == kMmaWarp || warp == kPvWarp) {
        // ---------------------------------------------------------------- MMA issuers
        // Two threads in different warps: one issues every S, the other every PV, both in
        // the stream's order. They share no operand, and each commit covers the MMAs of
        // the thread that makes it, so the two need no ordering between them.
        if (lane == 0) {
            auto k_desc = [&](int s) { return sdesc_sw128(sbase + C::kK + s * C::kTileBytes, 16, 1024); };
            auto v_desc = [&](int s) {
                return sdesc_sw128(sbase + C::kV + s * C::kTileBytes, C::kHalfBytes, 1024);
            };
            auto q_desc = [&](int b) {
                return sdesc_sw128(sbase + (F8 ? C::kQC + b * C::kQCBytes : C::kQ + b * C::kQBytes), 16, 1024);
            };
            auto p_desc = [&](int w) { return sdesc_sw128(sbase + C::kP + w * C::kPBytes, 16, 1024); };
            uint32_t g = 0, c[2] = {0, 0};  // tiles in all and of each warpgroup
            bool ok = true;
            const bool s_role = warp == kMmaWarp;
            for (int32_t q = 0; ok && item_of_round(2 * q) < total; ++q) {
                const int32_t nt[2] = {item_at(2 * q).nt,
                                       item_at(2 * q + 1).nt};
                const int32_t most = max(nt[0], nt[1]);
                for (int j = 0; j < most && ok; ++j) {
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        if (j >= nt[w] || !ok) continue;
                        if (s_role) {
                            // S^T = K Q^T: A = the K tile (K-major, 128 keys), B = Q^T (K-major,
                            // 16 rows); the S buffer is free once the tile before has its P
                            const int qb = q_buf(q, w);
                            if (j == 0 && !(ok = mbar_wait(q_full(qb), q_use(q), abort_flag))) break;
                            if (c[w] > 0 && !(ok = mbar_wait(p_full(w), (c[w] - 1) & 1, abort_flag))) break;
                            if (!(ok = mbar_wait(k_full(g % kKS), (g / kKS) & 1, abort_flag))) break;
                            tc_fence_after();
                            const uint64_t kd = k_desc(g % kKS), qd = q_desc(qb);
                            const uint32_t ts = tmem + C::kTmemS + w * kNS;
                            if constexpr (F8) {
#pragma unroll
                                for (int ks = 0; ks < kD / 32; ++ks)
                                    mma_ss_e4m3(ts, kd + (uint32_t)(ks * 2), qd + (uint32_t)(ks * 2), C::kIdescS,
                                                ks > 0 ? 1u : 0u);
                            } else {
#pragma unroll
                                for (int ks = 0; ks < kD / 16; ++ks) {
                                    const uint32_t koff = ((ks / 4) * C::kHalfBytes + (ks % 4) * 32) >> 4;
                                    const uint32_t qoff = ((ks / 4) * C::kRowsBytes + (ks % 4) * 32) >> 4;
                                    mma_ss(ts, kd + koff, qd + qoff, C::kIdescS, ks > 0 ? 1u : 0u);
                                }
                            }
                            mma_commit(s_full(w));
                            mma_commit(k_empty(g % kKS));
                            if (j + 1 == nt[w]) mma_commit(q_empty(qb));
                        } else {
                            // O^T = V^T P^T: A = the V tile read MN-major (M = D), B = P^T (K-major),
                            // once P is written, V is in and O of the tile before has been taken
                            if (!(ok = mbar_wait(p_full(w), c[w] & 1, abort_flag))) break;
                            if (!(ok = mbar_wait(v_full(g % kVS), (g / kVS) & 1, abort_flag))) break;
                            if (!(ok = mbar_wait(o_free(w), (c[w] & 1) ^ 1, abort_flag))) break;
                            tc_fence_after();
                            const uint64_t vd = v_desc(g % kVS), pd = p_desc(w);
                            const uint32_t to = tmem + C::kTmemO + w * kNO;
                            if constexpr (F8) {  // 32 keys (rows of 128 bytes of V, 32 bytes of P^T's) per MMA
#pragma unroll
                                for (int ks = 0; ks < kKeys / 32; ++ks)
                                    mma_ss_e4m3(to, vd + (uint32_t)(ks * 4096 >> 4), pd + (uint32_t)(ks * 2), C::kIdescO,
                                                ks > 0 ? 1u : 0u);
                            } else {
#pragma unroll
                                for (int ks = 0; ks < kKeys / 16; ++ks) {
                                    const uint32_t poff = ((ks / 4) * (kNO * 128) + (ks % 4) * 32) >> 4;
                                    mma_ss(to, vd + (uint32_t)(ks * 2048 >> 4), pd + poff, C::kIdescO,
                                           ks > 0 ? 1u : 0u);
                                }
                            }
                            mma_commit(o_full(w));
                            mma_commit(v_empty(g % kVS));
                        }
                        ++c[w];
                        ++g;
                    }
                }
            }
            if (!ok) report_status(a.status, PCP_ERR_TIMEOUT);
        }
    } else if (F8 && warp >= kConvWarp0) {
        // ---------------------------------------------------------------- e4m3: q terms
        const int cw = warp - kConvWarp0;
        bool ok = true;
        for (int32_t q = 0; ok && item_of_round(2 * q) < total; ++q) {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                if (item_of_round(2 * q + w) >= total) continue;
                const int qb = q_buf(q, w);
                if (!(ok = mbar_wait_warp(qc_full(qb), q_use(q), abort_flag))) break;
                if (q_to_e4m3_terms<GP>(smem + C::kQ + qb * C::kQBytes, smem + C::kQC + qb * C::kQCBytes,
                                        reinterpret_cast<float*>(smem + C::kQs) + qs_slot(q, w) * kGS, cw, lane, G) &&
                    lane == 0)
                    report_status(a.status, PCP_ERR_RANGE);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(q_full(qb));
                    mbar_arrive(q_ready(qs_slot(q, w)));
                }
            }
        }
        if (!ok && lane == 0) report_status(a.status, PCP_ERR_TIMEOUT);
    } else {
        // ---------------------------------------------------------------- softmax
        const int wg = warp / 4, wq = warp % 4;
        const int t = threadIdx.x % 128;  // key of the tile (S^T lane), dim (O^T lane)
        const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
        constexpr int kSpan = 32 / GP;     // lanes that end the reduce-scatter with one head
        const int hl = lane / kSpan;       // that head
        const uint32_t t_s = tmem + lane_base + C::kTmemS + wg * kNS;
        const uint32_t t_o = tmem + lane_base + C::kTmemO + wg * kNO;
        float* red_m = reinterpret_cast<float*>(smem + C::kRed) + wg * 2 * 4 * kGS;
        float* red_l = reinterpret_cast<float*>(smem + C::kSum) + wg * 2 * 4 * kGS;
        uint8_t* pbuf = smem + C::kP + wg * C::kPBytes;
        // this key's column of P^T: bf16: chunk (t % 64) / 8 of each row of half t / 64; e4m3:
        // chunk t / 16 of each row; swizzled by the row
        uint8_t* pcol = F8 ? pbuf + (t & 15) : pbuf + (t >> 6) * (kNO * 128) + (t & 7) * 2;
        const int chunk = F8 ? t >> 4 : (t & 63) >> 3;
        uint32_t gt = 0, c = 0;  // tiles of the stream before this pair, and this warpgroup's
        bool ok = true;     // every wait of this thread so far completed
        bool stop = false;  // the warpgroup's joint decision to stop, once per item
        for (int32_t q = 0; !stop && item_of_round(2 * q + wg) < total; ++q) {
            const PairItem it = item_at(2 * q + wg);
            const int32_t n_other = item_at(2 * q + 1 - wg).nt;
            const float kd = F8 ? __ldg(a.k_descale + (size_t)it.req * a.hkv + it.hk) : 1.f;
            const float sl2 = a.scale * kd * kLog2e;
            float sl2_pre = sl2, p_own = 1.f, p_pre = 1.f;
            if (F8 && it.preq != it.req) {
                const VScale f = v_scale(a, it);
                p_own = f.own;
                p_pre = f.pre;
                sl2_pre = a.scale * __ldg(a.k_descale + (size_t)it.preq * a.hkv + it.hk) * kLog2e;
            }
            // FP8: the power of two that undoes each head's q scaling (see q_to_e4m3_terms)
            float qs[GP];
#pragma unroll
            for (int h = 0; h < GP; ++h) qs[h] = 1.f;
            if constexpr (F8) {
                const int slot = qs_slot(q, wg);
                ok &= mbar_wait_warp(q_ready(slot), (q >> 2) & 1, abort_flag);
#pragma unroll
                for (int h = 0; h < GP; ++h) qs[h] = reinterpret_cast<const float*>(smem + C::kQs)[slot * kGS + h];
            }
            float m_run[GP], l_t[GP], acc[GP], a_prev[GP];
#pragma unroll
            for (int h = 0; h < GP; ++h) {
                m_run[h] = -INFINITY;
                l_t[h] = 0.f;
                acc[h] = 0.f;
                a_prev[h] = 0.f;
            }
            // O^T of this warpgroup's tile n (this thread's dim) into the running sums,
            // rescaled by the max update of that tile
            auto accumulate = [&](uint32_t n, const float (&alpha)[GP]) {
                ok &= mbar_wait_warp(o_full(wg), n & 1, abort_flag);
                tc_fence_after();
                uint32_t o[kNO];
                if constexpr (kNO == 32) {
                    tmem_ld32(t_o, o);
                } else {
                    tmem_ld16(t_o, o);
                }
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(o_free(wg));
#pragma unroll
                for (int h = 0; h < GP; ++h) {
                    const float o0 = __uint_as_float(o[h]), o1 = __uint_as_float(o[kTS + h]);
                    if constexpr (F8)  // the terms' powers of two taken back
                        acc[h] = acc[h] * alpha[h] + (o0 * 0x1p-8f + (o1 * 0x1p-12f + __uint_as_float(o[2 * kTS + h]) * 0x1p-16f));
                    else
                        acc[h] = acc[h] * alpha[h] + (o0 + o1);
                }
            };
            for (int j = 0; j < it.nt; ++j, ++c) {
                const int32_t v0 = it.lo + j * kKeys;
                const int nvalid = min(kKeys, it.hi - v0);
                const bool valid = t < nvalid && it.live(v0 + t);
                const bool pre = F8 && v0 + t < it.sinks;
                const float p_up = 0x1p8f * (pre ? p_pre : p_own);
                ok &= mbar_wait_warp(s_full(wg), c & 1, abort_flag);
                tc_fence_after();
                uint32_t s[kNS];
                tmem_ld16(t_s, s);
                tmem_wait_ld();
                float x[GP];
#pragma unroll
                for (int h = 0; h < GP; ++h) {
                    float sh = __uint_as_float(s[h]);
                    if constexpr (F8) {  // the q terms' scores, then the head's q scale
                        sh = (sh + __uint_as_float(s[GP + h])) * qs[h];
                    }
                    x[h] = valid ? sh * (pre ? sl2_pre : sl2) : -INFINITY;
                }
                // tile max per head: over the warp, then over the warpgroup's four warps
                float* rm = red_m + (c & 1) * 4 * kGS;  // [warp][head]
                const float wm = warp_scatter<GP, true>(x, lane);
                if (lane % kSpan == 0) rm[wq * kGS + hl] = wm;
                bar_sync_named(1 + wg, 128);
                // the tile before's O out of TMEM first: its PV complete frees the P buffer
                if (j > 0) accumulate(c - 1, a_prev);
#pragma unroll
                for (int h = 0; h < GP; ++h) {
                    const float mt = fmaxf(fmaxf(rm[h], rm[kGS + h]), fmaxf(rm[2 * kGS + h], rm[3 * kGS + h]));
                    const float m_new = fmaxf(m_run[h], mt);  // finite: every page read holds a key the row sees
                    const float alpha = fast_exp2(m_run[h] - m_new);  // 0 on the item's first tile
                    m_run[h] = m_new;
                    const float pe = fast_exp2(x[h] - m_new);
                    l_t[h] = l_t[h] * alpha + pe;
                    a_prev[h] = alpha;
                    if constexpr (F8) {
                        float term = pe * p_up;  // p 2^8, then the remainders 2^12 and 2^16
#pragma unroll
                        for (int n = 0; n < 3; ++n) {
                            const uint32_t code = f32x2_to_e4m3x2(term, 0.f);
                            const int row = n * kTS + h;
                            pcol[row * 128 + ((chunk ^ (row & 7)) << 4)] = (uint8_t)code;
                            if (n < 2) {
                                float back[4];
                                e4m3x4_to_f32(code, back);
                                term = (term - back[0]) * 16.f;  // exact: both hold few significant bits
                            }
                        }
                    } else {
                        const uint16_t hi = to16<F8>(pe);
                        const uint16_t lo = to16<F8>(pe - from16<F8>(hi));
                        *reinterpret_cast<uint16_t*>(pcol + h * 128 + ((chunk ^ (h & 7)) << 4)) = hi;
                        *reinterpret_cast<uint16_t*>(pcol + (kTS + h) * 128 + ((chunk ^ (h & 7)) << 4)) = lo;
                    }
                }
                // keys that the row does not see: zero their V rows (cache rows before the window,
                // unwritten slots of the last page, stale rows after it) once the tile has landed
                const bool gaps = nvalid < kKeys || (v0 < it.gap_end && it.gap_end > it.sinks);
                if (gaps) {
                    const uint32_t both = min(it.nt, n_other);  // tiles at which the stream alternates
                    const uint32_t g = gt + (j < (int)both ? 2 * j + wg : both + j), vs = g % kVS;
                    ok &= mbar_wait_warp(v_full(vs), (g / kVS) & 1, abort_flag);
                    if (!valid) {
                        uint8_t* vrow = smem + C::kV + vs * C::kTileBytes + t * 128;
#pragma unroll
                        for (int h = 0; h < (F8 ? 1 : 2); ++h)
#pragma unroll
                            for (int c2 = 0; c2 < 8; ++c2)
                                *reinterpret_cast<uint4*>(vrow + h * C::kHalfBytes + ((c2 ^ (t & 7)) << 4)) =
                                    make_uint4(0, 0, 0, 0);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(wg));
            }
            accumulate(c - 1, a_prev);
            gt += it.nt + n_other;
            float* rl = red_l + (q & 1) * 4 * kGS;  // [warp][head]
            const float wl = warp_scatter<GP, false>(l_t, lane);
            if (lane % kSpan == 0) rl[wq * kGS + hl] = wl;
            const float vd = F8 ? v_scale(a, it).all : 1.f;
            if ((stop = bar_wg_or(1 + wg, !ok))) break;
            if (a.cluster) {  // the split's sums for the cluster's merge, where its maxima and P were
                float* part = reinterpret_cast<float*>(pbuf);
#pragma unroll
                for (int h = 0; h < GP; ++h) {
                    part[h * kD + t] = acc[h];
                    if (t == 0) {
                        red_m[h] = m_run[h];
                        red_m[kGS + h] = rl[h] + rl[kGS + h] + rl[2 * kGS + h] + rl[3 * kGS + h];
                    }
                }
                continue;
            }
#pragma unroll
            for (int h = 0; h < GP; ++h) {
                if (h >= G) continue;
                const float L = rl[h] + rl[kGS + h] + rl[2 * kGS + h] + rl[3 * kGS + h];
                const float o = L > 0.f ? acc[h] / L * vd : 0.f;
                const float lse = L > 0.f ? (m_run[h] + __log2f(L)) * kLn2 : -INFINITY;
                const int32_t head = it.hk * G + h;
                if (a.direct) {
                    reinterpret_cast<__nv_bfloat16*>(a.out)[((size_t)it.q_start * a.hq + head) * kD + t] =
                        __float2bfloat16_rn(o);
                    if (t == 0) a.lse[(size_t)head * a.total_q + it.q_start] = lse;
                } else {
                    const size_t slot = ((size_t)it.row * a.hq + head) * max_splits + it.lo / a.chunk;
                    dec_out[slot * kD + t] = o;
                    if (t == 0) dec_lse[slot] = lse;
                }
            }
        }
        if (stop && t == 0) report_status(a.status, PCP_ERR_TIMEOUT);
    }

    __syncwarp();  // lane 0 of the MMA warps and of the producers worked alone: reconverge first
    if (a.cluster) {
        // the row's splits joined: head h by warpgroup h of the cluster (mod their number), a dim
        // per thread, reading the sums of split s where warpgroup s % 2 of block s / 2 left them
        cluster_sync();
        const int32_t n = *row_splits;
        if (warp < 8 && n > 0) {
            const int wg = warp / 4, t = threadIdx.x % 128;
            const PairItem it = own[0];
            const float vd = F8 ? v_scale(a, it).all : 1.f;
            const int32_t rank = (int32_t)blockIdx.x % a.cluster;
            for (int h = 2 * rank + wg; h < G; h += 2 * a.cluster) {
                float m[2 * kMaxCluster], l[2 * kMaxCluster], x[2 * kMaxCluster];
#pragma unroll
                for (int s = 0; s < 2 * kMaxCluster; ++s) {
                    m[s] = -INFINITY;
                    l[s] = x[s] = 0.f;
                    if (s >= n) continue;
                    const uint32_t at = sbase + C::kRed + (s & 1) * 2 * 4 * kGS * 4 + h * 4;
                    m[s] = cluster_load(at, s >> 1);
                    l[s] = cluster_load(at + kGS * 4, s >> 1);
                    x[s] = cluster_load(sbase + C::kP + (s & 1) * C::kPBytes + (h * kD + t) * 4, s >> 1);
                }
                float M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
                for (int s = 0; s < 2 * kMaxCluster; ++s) M = fmaxf(M, m[s]);
#pragma unroll
                for (int s = 0; s < 2 * kMaxCluster; ++s) {
                    const float f = s < n ? fast_exp2(m[s] - M) : 0.f;
                    L += f * l[s];
                    O += f * x[s];
                }
                const int32_t head = it.hk * G + h;
                reinterpret_cast<__nv_bfloat16*>(a.out)[((size_t)it.q_start * a.hq + head) * kD + t] =
                    __float2bfloat16_rn(L > 0.f ? O / L * vd : 0.f);
                if (t == 0) a.lse[(size_t)head * a.total_q + it.q_start] = L > 0.f ? (M + __log2f(L)) * kLn2 : -INFINITY;
            }
        }
        __syncwarp();
        cluster_sync();  // no block ends while another still reads its shared memory
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

template <bool F8, int GP>
int launch_pair(const PrefillArgs& a, float* dec_out, float* dec_lse, int32_t max_splits, cudaStream_t stream) {
    const int64_t slots = a.num_blocks * a.block_size;
    const int q_rows = a.hq < kN ? a.hq : kN;
    CUtensorMap tq, tk, tv;
    bool maps = make_box_map(&tq, a.q, kD, 2, a.hq, a.total_q, 64, q_rows, 1, true);
    if (F8)
        maps = maps && make_box_map(&tk, a.key_cache, kD, 1, a.hkv, slots, kD, 1, a.block_size, true) &&
               make_box_map(&tv, a.value_cache, kD, 1, a.hkv, slots, kD, 1, a.block_size, true);
    else
        maps = maps && make_box_map(&tk, a.key_cache, kD, 2, a.hkv, slots, 64, 1, a.block_size, true) &&
               make_box_map(&tv, a.value_cache, kD, 2, a.hkv, slots, 64, 1, a.block_size, true);
    if (!maps) return PCP_ERR_CUDA;
    const int smem = PairCfg<F8, GP>::kSmem;
    cudaError_t e =
        cudaFuncSetAttribute(decode_pair_kernel<F8, GP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) {
        if (a.cluster) {
            e = launch_clusters((unsigned)a.cluster, decode_pair_kernel<F8, GP>, dim3(a.num_rows * a.hkv * a.cluster),
                                dim3(PairCfg<F8, GP>::kThreads), smem, stream, tq, tk, tv, a, dec_out, dec_lse, max_splits,
                                q_rows);
        } else if (a.inline_items) {  // nothing of this call to be chained behind
            decode_pair_kernel<F8, GP><<<a.num_sms, PairCfg<F8, GP>::kThreads, smem, stream>>>(tq, tk, tv, a, dec_out, dec_lse,
                                                                                      max_splits, q_rows);
            e = cudaGetLastError();
        } else {
            e = launch_chained(decode_pair_kernel<F8, GP>, dim3(a.num_sms), dim3(PairCfg<F8, GP>::kThreads), smem, stream, tq,
                               tk, tv, a, dec_out, dec_lse, max_splits, q_rows);
        }
    }
    if (e != cudaSuccess) { set_last_cuda_error(e); return PCP_ERR_CUDA; }
    return PCP_OK;
}

}  // namespace

bool decode_inline_applies(const PrefillArgs& a, int32_t max_splits) {
    return decode_tc_applies(a) && a.num_prefixes == 0 && a.total_q <= a.num_rows && a.num_rows <= kInlineRows &&
           (int64_t)a.num_rows * a.hkv * max_splits <= 2 * a.num_sms;
}

// Blocks per row and kv head of a call whose one-token rows (as many as tokens) a
// cluster each can take side by side; 0: none. max_splits and a.chunk: the splits that the
// call would have otherwise.
// Clusters that all run at once: 15 of 8 blocks, 36 of 4, 76 of 2 fit the 152 SMs (one
// more and 1024-key windows take 18.5 us instead of 11.1, 22.6 instead of 14.3), a few
// are left for GPCs with fewer SMs. Where they leave SMs idle, their splits are at most one
// tile longer than those that a call with a merge would have: a row of 16452 slots and
// one kv head takes 27.4 us in one cluster, 22.6 with 304 splits and a merge (but 64
// such pairs of a row and a head, two blocks each, 85 against 95). One split per
// row (max_splits 1) needs no joining.
// With shared prefixes every row reads its prefix itself, most of it from L2: with 2 to 32
// rows, 1 to 8 kv heads and a bf16 cache 12 to 14 us instead of 23 to 25 behind 256 keys, 12 to 20
// instead of 24 to 28 behind 1008, 25 to 27 instead of 28 to 37 with 1000 keys per split, 41
// instead of 36 to 40 with 2000 (e4m3: 12 to 20 instead of 25 to 29 behind 1008 keys).
int32_t decode_cluster(const PrefillArgs& a, int64_t max_len, int32_t max_splits) {
    if (!decode_tc_applies(a) || a.total_q > a.num_rows || (max_splits == 1 && a.num_prefixes == 0)) return 0;
    if (a.num_prefixes > kClusterGroups) return 0;
    const int64_t units = (int64_t)a.num_rows * a.hkv;
    for (int32_t c = kMaxCluster; c >= 1; c /= 2) {
        if ((units + 5) * c > a.num_sms) continue;
        const int64_t keys = (max_len + 2 * c * kKeys - 1) / (2 * c * kKeys) * kKeys;
        if (a.num_prefixes > 0) return keys <= kPrefixKeys ? c : 0;
        return units * c * 4 >= a.num_sms * 3 || keys <= a.chunk + kKeys ? c : 0;
    }
    return 0;
}

int launch_decode_pair(const PrefillArgs& a, float* dec_out, float* dec_lse, int32_t max_splits,
                       cudaStream_t stream) {
    if (!decode_tc_applies(a)) return PCP_ERR_UNSUPPORTED;
    const int G = a.hq / a.hkv;
    // heads per group padded to a power of two (the padded heads' results are not written)
    const int GP = G <= 1 ? 1 : G <= 2 ? 2 : G <= 4 ? 4 : G <= 8 ? 8 : 16;
    if (a.k_descale) {
        if (GP == 1) return launch_pair<true, 1>(a, dec_out, dec_lse, max_splits, stream);
        if (GP == 2) return launch_pair<true, 2>(a, dec_out, dec_lse, max_splits, stream);
        if (GP == 4) return launch_pair<true, 4>(a, dec_out, dec_lse, max_splits, stream);
        return launch_pair<true, 8>(a, dec_out, dec_lse, max_splits, stream);
    }
    if (GP == 1) return launch_pair<false, 1>(a, dec_out, dec_lse, max_splits, stream);
    if (GP == 2) return launch_pair<false, 2>(a, dec_out, dec_lse, max_splits, stream);
    if (GP == 4) return launch_pair<false, 4>(a, dec_out, dec_lse, max_splits, stream);
    if (GP == 8) return launch_pair<false, 8>(a, dec_out, dec_lse, max_splits, stream);
    return launch_pair<false, 16>(a, dec_out, dec_lse, max_splits, stream);
}

}  // namespace pcp
