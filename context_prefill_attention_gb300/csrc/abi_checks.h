// Argument checks that the entry points share (host).
#pragma once

#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "pcp.h"

namespace pcp {

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// A device buffer as a byte range.
struct Span {
    const void* p;
    size_t n;
};

// True when two byte ranges share a byte (an empty range shares none).
inline bool overlap(Span a, Span b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.n > 0 && b.n > 0 && x < y + b.n && y < x + a.n;
}

// True when an output range overlaps any of the ranges in ins[0, n) (kernels
// read their inputs while other CTAs already write their outputs).
inline bool overlaps_any(Span out, const Span* ins, int n) {
    for (int i = 0; i < n; ++i)
        if (overlap(out, ins[i])) return true;
    return false;
}

// The sizes, scale and shape limits of an attention call (flags_ok: its flags
// are valid).
inline int check_attn_shape(int32_t num_reqs, int32_t max_blocks_per_req, int64_t num_blocks, int32_t block_size,
                            int32_t num_rows, int32_t total_q, int32_t num_q_heads, int32_t num_kv_heads,
                            int32_t head_dim, float scale, bool flags_ok) {
    if (num_rows < 0 || total_q < 0 || num_reqs < 0 || num_q_heads < 1 || num_kv_heads < 1 || max_blocks_per_req < 0 ||
        num_blocks < 0 || block_size < 1)
        return PCP_ERR_ARG;
    if (!flags_ok || !isfinite(scale)) return PCP_ERR_ARG;
    if (num_q_heads % num_kv_heads != 0) return PCP_ERR_UNSUPPORTED;
    if (head_dim != 64 && head_dim != 128) return PCP_ERR_UNSUPPORTED;
    if (block_size != 8 && block_size != 16 && block_size != 32 && block_size != 64 && block_size != 128)
        return PCP_ERR_UNSUPPORTED;
    if (num_q_heads / num_kv_heads > 16) return PCP_ERR_UNSUPPORTED;
    return PCP_OK;
}

}  // namespace pcp
