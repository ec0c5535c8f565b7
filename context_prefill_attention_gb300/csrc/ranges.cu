// Entry points of the attention calls over part of each row's keys: a sliding
// window with sinks (pcp_attn_window) and a batch that shares prefixes
// (pcp_attn_shared_prefix). Argument checks, workspace layout and the launch
// sequence; the kernels are in attn_prefill.cu (packed tiles of tokens x q
// heads), attn_decode_pair.cu and attn_decode.cu (one-token rows, the merge).
#include <cuda_runtime.h>
#include <stdint.h>

#include "abi_checks.h"
#include "pcp.h"
#include "pcp_internal.h"

namespace pcp {

namespace {

constexpr int kSms = 152;          // SMs the work is split for (the sizes of a call must not depend on a device)
constexpr int kMaxPrefixes = 1024;
constexpr int kMaxShards = 32;     // shards of a prefix

struct RangeLayout {
    size_t header, row_ok, row_lo, merge, dec_units, units, units_sorted, part_out, part_lse, dec_out,
        dec_lse, total;
    int64_t max_units;
    int32_t slots, chunk, max_splits, nparts;
};

// Keys per decode split (a multiple of 128, at most kDecodeChunk): the length with
// the shortest modelled time for rows of max_len slots. An SM takes its share of
// the items two at a time; a pair takes about 3 us to start and end, and a tile
// of each 1.5 us by latency, 2.9 us once every SM draws on HBM; every split
// is one more partial to merge.
int32_t decode_chunk(int32_t num_rows, int32_t hkv, int64_t max_len) {
    const int64_t items = (int64_t)num_rows * hkv;
    double best = 0;
    int32_t best_chunk = kDecodeChunk;
    for (int32_t c = kDecodeChunk; c >= kBlockN; c -= kBlockN) {
        const int64_t splits = (max_len + c - 1) / c;
        const int64_t tiles = ((max_len < c ? max_len : c) + kBlockN - 1) / kBlockN;
        const double pairs = (double)(items * splits) / (2 * kSms);
        const double tile_us = 1.5 + 1.4 * (pairs < 1 ? pairs : 1);
        const double t = (double)(int64_t)(pairs + 0.9999) * (3 + (double)tiles * tile_us) + 0.3 * (double)splits;
        if (c == kDecodeChunk || t < best) {
            best = t;
            best_chunk = c;
        }
    }
    return best_chunk;
}

// The most shards of a prefix (its partials take workspace; the scheduler picks how
// many): enough to give every SM four items.
int32_t most_shards(int32_t total_q, int32_t hkv, int32_t span, int64_t max_kv) {
    const int64_t items = (total_q + span - 1) / span * (int64_t)hkv;
    const int64_t tiles = (max_kv + kBlockN - 1) / kBlockN;
    int64_t n = items > 0 ? (4 * kSms + items - 1) / items + 1 : 1;
    if (n > tiles / 2) n = tiles / 2;
    if (n > kMaxShards) n = kMaxShards;
    return n > 1 ? (int32_t)n : 1;
}

// num_prefixes < 0: a window call.
RangeLayout range_layout(int32_t num_rows, int32_t num_prefixes, int32_t total_q, int32_t hq, int32_t hkv, int32_t d,
                         int64_t max_kv, int64_t max_len) {
    RangeLayout w{};
    const int32_t tpt = kBlockM / (hq / hkv);
    w.slots = total_q > tpt ? 2 : 1;
    const int32_t span = w.slots * tpt;
    w.chunk = decode_chunk(num_rows, hkv, max_len);
    w.max_splits = max_len > 0 ? (int32_t)((max_len + w.chunk - 1) / w.chunk) : 1;
    const int32_t ng = num_prefixes > 0 ? num_prefixes : 0;
    const int32_t shards = ng > 0 ? most_shards(total_q, hkv, span, max_kv) : 0;
    w.nparts = ng > 0 ? shards + 1 : 0;
    const int64_t tiles = (total_q + span - 1) / span;
    w.max_units = tiles + num_rows + shards * (tiles + ng);
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o = align256(o + bytes);
        return at;
    };
    w.header = take(64 * sizeof(int32_t));
    w.row_ok = take((size_t)num_rows * 4);
    w.row_lo = take((size_t)num_rows * 4);
    w.merge = take((size_t)(ng > 0 ? total_q : num_rows) * sizeof(MergeTask));
    w.dec_units = take(num_rows <= kDecTcMaxRows ? (size_t)num_rows * w.max_splits * sizeof(DecUnit) : 0);
    w.units = take((size_t)w.max_units * sizeof(PackedUnit));
    w.units_sorted = take((size_t)w.max_units * sizeof(PackedUnit));
    w.part_out = take((size_t)w.nparts * total_q * hq * d * 4);
    w.part_lse = take((size_t)w.nparts * total_q * hq * 4);
    const size_t dec = (size_t)num_rows * hq * w.max_splits;
    w.dec_out = take(dec * d * 4);
    w.dec_lse = take(dec * 4);
    w.total = o;
    return w;
}

// Workspace for a call of up to num_rows rows, num_prefixes groups and total_q tokens:
// a smaller call can be split finer, so the parts that grow with the splits are
// taken at their largest over all smaller calls (a caller sizes its workspace once).
size_t range_workspace(int32_t num_rows, int32_t num_prefixes, int32_t total_q, int32_t hq, int32_t hkv, int32_t d,
                       int64_t max_kv, int64_t max_len) {
    const RangeLayout w = range_layout(num_rows, num_prefixes, total_q, hq, hkv, d, max_kv, max_len);
    // decode partials and records: rows x splits
    int64_t splits = (int64_t)num_rows * w.max_splits, most_splits = splits;
    for (int32_t r = 1; r < num_rows; ++r) {
        const int32_t c = decode_chunk(r, hkv, max_len);
        const int64_t n = (int64_t)r * (max_len > 0 ? (max_len + c - 1) / c : 1);
        if (n > most_splits) most_splits = n;
    }
    // partials of the prefixes and units: they change with the tokens' tiles, of one or two per item
    int64_t parts = (int64_t)w.nparts * total_q, most_parts = parts, most_units = w.max_units;
    const int32_t tpt = kBlockM / (hq / hkv);
    for (int64_t t = tpt; t < total_q; t += tpt) {
        const RangeLayout x = range_layout(0, num_prefixes, (int32_t)t, hq, hkv, d, max_kv, 0);
        if ((int64_t)x.nparts * t > most_parts) most_parts = (int64_t)x.nparts * t;
        if (x.max_units + num_rows > most_units) most_units = x.max_units + num_rows;
    }
    return w.total + (size_t)(most_splits - splits) * ((size_t)hq * (d + 1) * 4 + sizeof(DecUnit)) +
           (size_t)(most_parts - parts) * hq * (d + 1) * 4 +
           (size_t)(most_units - w.max_units) * 2 * sizeof(PackedUnit) + 16 * 256;
}

// Slots of the longest walk of a one-token row (KeyRange::len).
int64_t window_len(int64_t max_kv, int32_t block_size, int32_t window, int32_t sinks) {
    const int64_t n = (int64_t)window + sinks + 2 * block_size;
    return n < max_kv ? n : max_kv;
}

struct RangeCall {
    const void *q, *key_cache, *value_cache;
    const float *k_descale, *v_descale;
    const int32_t* block_table;
    int32_t num_reqs, max_blocks;
    int64_t num_blocks;
    int32_t block_size;
    const pcp_row_t* rows;
    int32_t num_rows, total_q, hq, hkv, d;
    float scale;
    void* out;
    float* lse;
    void* workspace;
    size_t workspace_bytes;
    int32_t* status;
    cudaStream_t stream;
    bool fp8;
    int32_t window, sinks;
    const pcp_prefix_t* prefixes;
    int32_t num_prefixes;  // -1: a window call
};

int range_call(const RangeCall& c) {
    const int shape = check_attn_shape(c.num_reqs, c.max_blocks, c.num_blocks, c.block_size, c.num_rows, c.total_q,
                                       c.hq, c.hkv, c.d, c.scale, true);
    if (shape != PCP_OK) return shape;
    if (c.num_rows == 0 || c.total_q == 0) return PCP_OK;
    if (!c.q || !c.key_cache || !c.value_cache || !c.block_table || !c.rows || !c.out || !c.lse || !c.workspace ||
        (c.fp8 && (!c.k_descale || !c.v_descale)) || (c.num_prefixes > 0 && !c.prefixes))
        return PCP_ERR_ARG;
    if (!aligned16(c.q) || !aligned16(c.key_cache) || !aligned16(c.value_cache) || !aligned16(c.out) ||
        !aligned4(c.lse) || (reinterpret_cast<uintptr_t>(c.workspace) & 255u) || !aligned4(c.block_table) ||
        !aligned4(c.rows) || !aligned4(c.k_descale) || !aligned4(c.v_descale) || !aligned4(c.prefixes))
        return PCP_ERR_ALIGN;
    if (c.num_blocks * (int64_t)c.block_size > INT32_MAX || (int64_t)c.total_q * c.hq > INT32_MAX) return PCP_ERR_ARG;
    const int64_t max_kv = (int64_t)c.max_blocks * c.block_size;
    if (max_kv > INT32_MAX - 1024) return PCP_ERR_ARG;  // positions are rounded up to tiles and pages in 32 bits
    const bool shared = c.num_prefixes >= 0;
    const int64_t max_len = shared ? max_kv : window_len(max_kv, c.block_size, c.window, c.sinks);
    const RangeLayout w = range_layout(c.num_rows, c.num_prefixes, c.total_q, c.hq, c.hkv, c.d, max_kv, max_len);
    if (c.workspace_bytes < w.total) return PCP_ERR_WORKSPACE;
    const size_t out_bytes = (size_t)c.total_q * c.hq * c.d * 2, lse_bytes = (size_t)c.total_q * c.hq * 4;
    const size_t cache_bytes = (size_t)c.num_blocks * c.block_size * c.hkv * c.d * (c.fp8 ? 1 : 2);
    const size_t descale_bytes = c.fp8 ? (size_t)c.num_reqs * c.hkv * 4 : 0;
    const Span ins[9] = {{c.q, out_bytes},
                         {c.key_cache, cache_bytes},
                         {c.value_cache, cache_bytes},
                         {c.block_table, (size_t)c.num_reqs * c.max_blocks * 4},
                         {c.rows, (size_t)c.num_rows * sizeof(pcp_row_t)},
                         {c.workspace, w.total},
                         {c.k_descale, descale_bytes},
                         {c.v_descale, descale_bytes},
                         {c.prefixes, shared ? (size_t)c.num_prefixes * sizeof(pcp_prefix_t) : 0}};
    if (overlaps_any({c.out, out_bytes}, ins, 9) || overlaps_any({c.lse, lse_bytes}, ins, 9) ||
        overlap({c.out, out_bytes}, {c.lse, lse_bytes}))
        return PCP_ERR_ARG;

    uint8_t* ws = static_cast<uint8_t*>(c.workspace);
    auto ints = [&](size_t at) { return reinterpret_cast<int32_t*>(ws + at); };
    PrefillArgs a{};
    a.q = c.q;
    a.key_cache = c.key_cache;
    a.value_cache = c.value_cache;
    a.block_table = c.block_table;
    a.num_reqs = c.num_reqs;
    a.max_blocks = c.max_blocks;
    a.num_blocks = c.num_blocks;
    a.block_size = c.block_size;
    a.rows = c.rows;
    a.num_rows = c.num_rows;
    a.total_q = c.total_q;
    a.hq = c.hq;
    a.hkv = c.hkv;
    a.d = c.d;
    a.scale = c.scale;
    a.out = c.out;
    a.lse = c.lse;
    a.part_out = reinterpret_cast<float*>(ws + w.part_out);
    a.part_lse = reinterpret_cast<float*>(ws + w.part_lse);
    a.nparts = w.nparts;
    a.row_ok = ints(w.row_ok);
    a.packed = reinterpret_cast<const PackedUnit*>(ws + w.units_sorted);
    a.num_units = ints(w.header);
    a.dec_units = reinterpret_cast<const DecUnit*>(ws + w.dec_units);
    a.status = c.status;
    a.k_descale = c.fp8 ? c.k_descale : nullptr;
    a.v_descale = c.fp8 ? c.v_descale : nullptr;
    a.chunk = w.chunk;
    a.window = c.window;
    a.sinks = c.sinks;
    a.slots = w.slots;
    a.row_lo = ints(w.row_lo);
    a.prefixes = c.prefixes;
    a.num_prefixes = shared ? c.num_prefixes : 0;

    a.num_sms = num_sms();
    a.overlap = decode_tc_applies(a);
    a.direct = !shared && w.max_splits == 1;
    MergeTask* tasks = reinterpret_cast<MergeTask*>(ws + w.merge);
    a.merge = tasks;
    a.cluster = decode_cluster(a, max_len, w.max_splits);
    a.inline_items = a.cluster > 0 || decode_inline_applies(a, w.max_splits);
    int rc = PCP_OK;
    if (!a.inline_items)
        rc = launch_range_schedule(a, reinterpret_cast<PackedUnit*>(ws + w.units),
                                   reinterpret_cast<PackedUnit*>(ws + w.units_sorted), ints(w.header), ints(w.row_ok),
                                   ints(w.row_lo), tasks, reinterpret_cast<DecUnit*>(ws + w.dec_units), w.max_units,
                                   c.stream);
    if (rc != PCP_OK) return rc;
    float* dec_out = reinterpret_cast<float*>(ws + w.dec_out);
    float* dec_lse = reinterpret_cast<float*>(ws + w.dec_lse);
    rc = launch_range_decode(a, dec_out, dec_lse, w.max_splits, c.stream);
    if (rc != PCP_OK) return rc;
    // no row can have two tokens when there are as many rows as tokens (the rows'
    // tokens are disjoint): only prefixes are left for the packed kernel
    if (c.total_q > c.num_rows || (a.num_prefixes > 0 && a.cluster == 0)) {
        rc = launch_packed(a, c.stream);
        if (rc != PCP_OK) return rc;
    }
    if (a.direct || a.cluster > 0) return PCP_OK;
    return launch_range_merge(a, tasks, dec_out, dec_lse, w.max_splits, c.stream);
}

bool window_ok(int32_t window, int32_t sinks) { return window >= 1 && sinks >= 0; }

}  // namespace

}  // namespace pcp

using namespace pcp;

extern "C" size_t pcp_attn_window_workspace_size(int32_t num_rows, int32_t total_q, int32_t num_q_heads,
                                                 int32_t num_kv_heads, int32_t head_dim, int32_t max_kv_len,
                                                 int32_t block_size, int32_t window, int32_t num_sinks) {
    if (num_rows < 0 || total_q < 0 || num_kv_heads < 1 || num_q_heads < num_kv_heads || num_q_heads % num_kv_heads ||
        num_q_heads / num_kv_heads > 16 || head_dim < 1 || max_kv_len < 0 || block_size < 1 ||
        !window_ok(window, num_sinks))
        return 0;
    return range_workspace(num_rows, -1, total_q, num_q_heads, num_kv_heads, head_dim, max_kv_len,
                           window_len(max_kv_len, block_size, window, num_sinks));
}

extern "C" size_t pcp_attn_shared_prefix_workspace_size(int32_t num_rows, int32_t num_prefixes, int32_t total_q,
                                                        int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                                        int32_t max_kv_len) {
    if (num_rows < 0 || num_prefixes < 0 || num_prefixes > kMaxPrefixes || total_q < 0 || num_kv_heads < 1 ||
        num_q_heads < num_kv_heads || num_q_heads % num_kv_heads || num_q_heads / num_kv_heads > 16 || head_dim < 1 ||
        max_kv_len < 0)
        return 0;
    return range_workspace(num_rows, num_prefixes, total_q, num_q_heads, num_kv_heads, head_dim, max_kv_len, max_kv_len);
}

extern "C" int pcp_attn_window(const void* q, const void* key_cache, const void* value_cache,
                               const int32_t* block_table, int32_t num_reqs, int32_t max_blocks_per_req,
                               int64_t num_blocks, int32_t block_size, const pcp_row_t* rows, int32_t num_rows,
                               int32_t total_q, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                               float scale, int32_t window, int32_t num_sinks, void* out, float* lse,
                               void* workspace, size_t workspace_bytes, int32_t* status, pcp_stream_t stream) {
    if (!window_ok(window, num_sinks)) return PCP_ERR_ARG;
    return range_call({q, key_cache, value_cache, nullptr, nullptr, block_table, num_reqs, max_blocks_per_req,
                       num_blocks, block_size, rows, num_rows, total_q, num_q_heads, num_kv_heads, head_dim, scale,
                       out, lse, workspace, workspace_bytes, status, reinterpret_cast<cudaStream_t>(stream), false,
                       window, num_sinks, nullptr, -1});
}

extern "C" int pcp_attn_window_fp8kv(const void* q, const void* key_cache, const void* value_cache,
                                     const float* k_descale, const float* v_descale, const int32_t* block_table,
                                     int32_t num_reqs, int32_t max_blocks_per_req, int64_t num_blocks,
                                     int32_t block_size, const pcp_row_t* rows, int32_t num_rows, int32_t total_q,
                                     int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, float scale,
                                     int32_t window, int32_t num_sinks, void* out, float* lse, void* workspace,
                                     size_t workspace_bytes, int32_t* status, pcp_stream_t stream) {
    if (!window_ok(window, num_sinks)) return PCP_ERR_ARG;
    return range_call({q, key_cache, value_cache, k_descale, v_descale, block_table, num_reqs, max_blocks_per_req,
                       num_blocks, block_size, rows, num_rows, total_q, num_q_heads, num_kv_heads, head_dim, scale,
                       out, lse, workspace, workspace_bytes, status, reinterpret_cast<cudaStream_t>(stream), true,
                       window, num_sinks, nullptr, -1});
}

extern "C" int pcp_attn_shared_prefix(const void* q, const void* key_cache, const void* value_cache,
                                      const int32_t* block_table, int32_t num_reqs, int32_t max_blocks_per_req,
                                      int64_t num_blocks, int32_t block_size, const pcp_row_t* rows,
                                      int32_t num_rows, const pcp_prefix_t* prefixes, int32_t num_prefixes,
                                      int32_t total_q, int32_t num_q_heads, int32_t num_kv_heads,
                                      int32_t head_dim, float scale, void* out, float* lse, void* workspace,
                                      size_t workspace_bytes, int32_t* status, pcp_stream_t stream) {
    if (num_prefixes < 0 || num_prefixes > kMaxPrefixes) return PCP_ERR_ARG;
    return range_call({q, key_cache, value_cache, nullptr, nullptr, block_table, num_reqs, max_blocks_per_req,
                       num_blocks, block_size, rows, num_rows, total_q, num_q_heads, num_kv_heads, head_dim, scale,
                       out, lse, workspace, workspace_bytes, status, reinterpret_cast<cudaStream_t>(stream), false,
                       INT32_MAX, 0, prefixes, num_prefixes});
}

extern "C" int pcp_attn_shared_prefix_fp8kv(const void* q, const void* key_cache, const void* value_cache,
                                            const float* k_descale, const float* v_descale,
                                            const int32_t* block_table, int32_t num_reqs,
                                            int32_t max_blocks_per_req, int64_t num_blocks, int32_t block_size,
                                            const pcp_row_t* rows, int32_t num_rows, const pcp_prefix_t* prefixes,
                                            int32_t num_prefixes, int32_t total_q, int32_t num_q_heads,
                                            int32_t num_kv_heads, int32_t head_dim, float scale, void* out,
                                            float* lse, void* workspace, size_t workspace_bytes, int32_t* status,
                                            pcp_stream_t stream) {
    if (num_prefixes < 0 || num_prefixes > kMaxPrefixes) return PCP_ERR_ARG;
    return range_call({q, key_cache, value_cache, k_descale, v_descale, block_table, num_reqs, max_blocks_per_req,
                       num_blocks, block_size, rows, num_rows, total_q, num_q_heads, num_kv_heads, head_dim, scale,
                       out, lse, workspace, workspace_bytes, status, reinterpret_cast<cudaStream_t>(stream), true,
                       INT32_MAX, 0, prefixes, num_prefixes});
}
