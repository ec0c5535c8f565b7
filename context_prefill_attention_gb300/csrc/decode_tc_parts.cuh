// Building blocks of the tensor-core decode kernels (attn_decode_tc.cu,
// attn_decode_pair.cu): roles, the converters' widening and q terms, and the
// softmax warps' reductions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "pcp_device.cuh"
#include "pcp_internal.h"

namespace pcp {

namespace {

constexpr int kD = 128;          // head_dim this kernel takes
constexpr int kKeys = 128;       // keys per tile: the M of S^T
constexpr int kN = 16;           // the N of S^T (and of O^T up to 8 q heads per kv head)
constexpr int kMaxG = 16;        // q heads per kv head (FP8: 8)
constexpr int kTerms = 2;        // FP8: e4m3 terms per q element (their sum is the bf16 q exactly)
constexpr int kProdWarp = 8;     // warp 8: K tiles and Q^T; warp 9: V tiles
constexpr int kMmaWarp = 10;     // lane 0 issues the S MMAs (the warp owns the TMEM allocation)
constexpr int kPvWarp = 11;      // lane 0 issues the PV MMAs
constexpr int kConvWarp0 = 12;
constexpr int kConvThreads = 128;  // FP8: threads widening one V tile (one or two such sets)
// FP8 converter warps: two sets of four taking alternate V tiles where the
// softmax fits the registers that 20 warps leave (G <= 4), else one set
__host__ __device__ constexpr int conv_warps(bool f8, int gp) { return f8 ? (gp <= 4 ? 8 : 4) : 0; }
__host__ __device__ constexpr int tc_threads(bool f8, int gp) { return 32 * (12 + conv_warps(f8, gp)); }
constexpr int kMaxPages = kDecodeChunk / 8;  // block-table entries of one split (block_size >= 8)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Named barrier `id` over `n` threads (whole warps).
__device__ __forceinline__ void bar_sync_named(int id, int n) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}

// Named barrier `id` over one softmax warpgroup (128 threads) that also ORs a
// predicate: every thread gets the same answer, so the warps leave their loops
// together.
__device__ __forceinline__ bool bar_wg_or(int id, bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)pred), "r"(id)
        : "memory");
    return r != 0;
}

// Max (kMax) or sum over the warp of GP values per lane, by reduce-scatter: each
// step with offset o = 16, 8, ... halves the values a lane keeps (the upper half
// where bit o of the lane is set), the remaining offsets reduce the last one.
// Lane l ends with head l / (32 / GP) reduced over all 32 lanes.
template <int GP, bool kMax>
__device__ __forceinline__ float warp_scatter(const float (&x)[GP], int lane) {
    float v[GP];
#pragma unroll
    for (int h = 0; h < GP; ++h) v[h] = x[h];
#pragma unroll
    for (int o = 16, n = GP; n > 1; o >>= 1, n >>= 1) {
        const bool upper = (lane & o) != 0;
#pragma unroll
        for (int k = 0; k < n / 2; ++k) {
            const float send = upper ? v[k] : v[k + n / 2];
            const float keep = upper ? v[k + n / 2] : v[k];
            const float r = __shfl_xor_sync(0xffffffffu, send, o);
            v[k] = kMax ? fmaxf(keep, r) : keep + r;
        }
    }
#pragma unroll
    for (int o = 16 / GP; o >= 1; o >>= 1) {
        const float r = __shfl_xor_sync(0xffffffffu, v[0], o);
        v[0] = kMax ? fmaxf(v[0], r) : v[0] + r;
    }
    return v[0];
}

// One tile of FP8 codes -> f16 in the 128-byte-swizzled K-major layout of a
// stage (dims 64h..64h+63 of row r in half h, 16-byte chunk c of that row at
// chunk c ^ (r & 7)). The codes of row r (128 bytes) sit where half 1 of row r
// goes; the eight threads of a row are in one warp and all load before any of
// them stores. Rows at or past nvalid are written as zeros (their codes may be
// stale or unwritten cache slots). Run by the 128 converter threads.
__device__ __forceinline__ void widen_tile(uint8_t* tile, int nvalid, int ct) {
    constexpr int kHalf = kKeys * 128;
    constexpr int kRpp = kConvThreads / 8;  // rows per pass
    constexpr int kBatch = 4;
    const int t = ct % 8, rsub = ct / 8;
    const int h = t / 4, c0 = 2 * (t % 4);
    // threads of the second half store their odd chunk first, so the eight
    // threads of a row hit eight different bank groups in each store
    const int first = c0 + (t >= 4 ? 1 : 0), second = c0 + (t >= 4 ? 0 : 1);
    const uint8_t* codes = tile + kHalf;
#pragma unroll 1
    for (int r0 = 0; r0 < kKeys; r0 += kRpp * kBatch) {
        uint4 c[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int r = r0 + kRpp * b + rsub;
            c[b] = r < nvalid ? *reinterpret_cast<const uint4*>(codes + r * kD + 16 * t)
                                         : make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int r = r0 + kRpp * b + rsub;
            const uint2 w0 = e4m3x4_to_f16x4(c[b].x), w1 = e4m3x4_to_f16x4(c[b].y);
            const uint2 w2 = e4m3x4_to_f16x4(c[b].z), w3 = e4m3x4_to_f16x4(c[b].w);
            const uint4 lo = make_uint4(w0.x, w0.y, w1.x, w1.y);  // dims 16t .. 16t+7
            const uint4 hi = make_uint4(w2.x, w2.y, w3.x, w3.y);  // dims 16t+8 .. 16t+15
            uint8_t* row = tile + h * kHalf + r * 128;
            const bool lo_first = first == c0;
            *reinterpret_cast<uint4*>(row + ((first ^ (r & 7)) << 4)) = lo_first ? lo : hi;
            *reinterpret_cast<uint4*>(row + ((second ^ (r & 7)) << 4)) = lo_first ? hi : lo;
        }
        __syncwarp();
    }
}

// FP8: the group's q heads as kTerms e4m3 terms each. Input: the bf16 Q^T
// tile as TMA wrote it (two 64-dim halves of 16 rows, 128-byte swizzled).
// Output: the swizzled K-major layout of an e4m3 MMA operand, row t * GP + h
// holding term t of head h (128 codes, 16-byte chunk c of row r at chunk
// c ^ (r & 7)). Head h is first scaled by 2^(8 - ex), ex the binary exponent
// of its largest magnitude (frexp), so that every element lies below 256. The
// first term is the e4m3 rounding of the scaled element x (4 significant bits);
// the remainder x - term is a multiple of x's last bit no larger than 8 of
// them (x has 8 significant bits), so it is an e4m3 value too and the two
// terms sum to x exactly, unless the remainder falls under e4m3's smallest
// subnormal (2^-9 of the scaled unit, where the largest element lies in
// [128, 256): only elements below 2^-9 of the head's largest can lose bits, at
// most 2^-17 of it). qscale[h] = 2^(ex - 8) undoes
// the scaling. Warp w of the converter set does heads w and w + 4, lane l dims
// 4l .. 4l + 3. Returns whether an element of one of the G real heads lies
// beyond +-65504 (reported as PCP_ERR_RANGE, as the prefill rows' q is).
template <int GP>
__device__ __forceinline__ bool q_to_e4m3_terms(const uint8_t* qbf, uint8_t* qc, float* qscale, int w, int lane,
                                                int G) {
    bool over = false;
#pragma unroll
    for (int h = w; h < GP; h += 4) {
        const int d = 4 * lane, half = d >> 6, col = d & 63;
        const uint2 raw =
            *reinterpret_cast<const uint2*>(qbf + half * (kN * 128) + h * 128 + (((col >> 3) ^ (h & 7)) << 4) + (col & 7) * 2);
        float x[4] = {__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xFFFF0000u),
                      __uint_as_float(raw.y << 16), __uint_as_float(raw.y & 0xFFFF0000u)};
        float m = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        over |= h < G && m > 65504.f;
        int ex = 0;
        frexpf(m, &ex);
        const float f = ldexpf(1.f, 8 - ex);
        if (lane == 0) qscale[h] = ldexpf(1.f, ex - 8);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] *= f;
#pragma unroll
        for (int t = 0; t < kTerms; ++t) {
            const uint32_t codes = f32x2_to_e4m3x2(x[0], x[1]) | (f32x2_to_e4m3x2(x[2], x[3]) << 16);
            const int row = t * GP + h;
            *reinterpret_cast<uint32_t*>(qc + row * 128 + (((d >> 4) ^ (row & 7)) << 4) + (d & 15)) = codes;
            if (t + 1 < kTerms) {
                float back[4];
                e4m3x4_to_f32(codes, back);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] -= back[e];  // exact: both hold few significant bits
            }
        }
    }
    return over;
}

template <bool F8>
__device__ __forceinline__ uint16_t to16(float x) {
    if constexpr (F8) return __half_as_ushort(__float2half_rn(x));
    return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}
template <bool F8>
__device__ __forceinline__ float from16(uint16_t x) {
    if constexpr (F8) return __half2float(__ushort_as_half(x));
    return __bfloat162float(__ushort_as_bfloat16(x));
}

}  // namespace

}  // namespace pcp
