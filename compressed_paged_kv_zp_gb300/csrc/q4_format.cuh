// q4_format.cuh -- the 4-bit cache: layout of a tile, and the arguments checks
// that its calls share.
//
// A tile holds 16 tokens of one kv head of one block: 16 rows of d/2 bytes of codes
// (element e in nibble e, low nibble first), then 16 rows of d/group words, one per
// group of elements: step (bf16) in the low half, lo (bf16) in the high half; the
// element's value is lo + code * step.  One layer is [N_total][h_kv][b/16][tile].
//
// The 16-byte chunks of a row's codes are exchanged by its token: chunk c of row t
// lies at c ^ ((t >> 1) & 3) (d = 128: two rows fill the 32 banks) or c ^ ((t >> 2) & 1)
// (d = 64: four rows do).  Any eight consecutive rows then have a given chunk in eight
// different 16-byte columns of a 128-byte line, so that ldmatrix reads a tile that was
// copied to shared memory as it is without bank conflicts.
#pragma once

#include "zp_common.cuh"

namespace zp {

constexpr int kQ4Tile = 16;         // tokens per tile
constexpr int kQ4MaxGroups = 4;     // groups per row: d/group
constexpr uint32_t kQ4NaN = 0x7FC07FC0u;  // step and lo of a group that holds anything not finite

__host__ __device__ constexpr int q4_code_bytes(int d) { return kQ4Tile * d / 2; }
__host__ __device__ constexpr int q4_tile_bytes(int d, int group) { return q4_code_bytes(d) + kQ4Tile * 4 * (d / group); }

template <int D>
__host__ __device__ __forceinline__ int q4_chunk(int t, int c) {
    return D == 128 ? (c ^ ((t >> 1) & 3)) : (c ^ ((t >> 2) & 1));
}

// bf16 bits of the largest bf16 value not above x, and of the smallest not below it
// (x not NaN; a result past the largest finite value is an infinity).
__device__ __forceinline__ uint32_t bf16_below(float x) {
    const uint32_t u = __float_as_uint(x);
    return ((u & 0xFFFFu) && (u >> 31) ? u + 0x10000u : u) >> 16;
}
__device__ __forceinline__ uint32_t bf16_above(float x) {
    const uint32_t u = __float_as_uint(x);
    return ((u & 0xFFFFu) && !(u >> 31) ? u + 0x10000u : u) >> 16;
}

// The word (step, lo) of a group whose smallest and largest element are mn and mx
// (NaN if one of its elements is): lo is the bf16 value at or below mn, the step the
// bf16 value at or above a fifteenth of mx - lo, so that fifteen steps reach mx and no
// element is further than half a step from its code's value.  For bf16 elements lo is
// mn itself.  The step is at least 2^-126 (its reciprocal is finite).
__device__ __forceinline__ uint32_t q4_params(float mn, float mx) {
    const uint32_t lo = bf16_below(mn);
    const float flo = __uint_as_float(lo << 16);
    const float step = fmaxf(__uint_as_float(bf16_above(__fdiv_rn(mx - flo, 15.f)) << 16), __uint_as_float(0x00800000u));
    const bool finite = fabsf(flo) < INFINITY && step < INFINITY && mx - flo < INFINITY;  // (a NaN compares false)
    return finite ? (__float_as_uint(step) >> 16) | (lo << 16) : kQ4NaN;
}

// Code of x in a group with (step, lo): floor((x - lo) / step + 1/2), the quotient not
// rounded.  r is a reciprocal of the step a little too small, so that t's integer k is
// the code or one less; x - lo - k * step is exact (k * step has 12 bits, the difference
// at most half a step) and tells which.  half = step / 2.
__device__ __forceinline__ uint32_t q4_code(float x, float lo, float step, float r, float half) {
    const float d = x - lo;
    const float t = fmaf(d, r, 12582912.f);  // 1.5 * 2^23: the integer in the low bits
    const float rest = fmaf(-(t - 12582912.f), step, d);
    return __float_as_uint(t) + (rest >= half ? 1u : 0u);  // the caller keeps the low 4 bits
}

__device__ __forceinline__ float q4_shrunk_reciprocal(float step) {
    return __fmul_rn(__frcp_rn(step), 1.f - 9.5367431640625e-7f);  // 1 - 2^-20
}

// Host: arguments that every call on a 4-bit cache has.
inline zp_status check_q4(const zp_cache_desc *D, int group, const char *what) {
    const zp_status rc = check_desc(D);
    if (rc != ZP_OK) return rc;
    if (D->head_dim != 64 && D->head_dim != 128) return fail(ZP_ERR_SHAPE, "%s: head_dim %d", what, D->head_dim);
    if (group != 32 && group != 64 && group != 128) return fail(ZP_ERR_SHAPE, "%s: group %d", what, group);
    if (group > D->head_dim) return fail(ZP_ERR_SHAPE, "%s: group %d above head_dim %d", what, group, D->head_dim);
    if (D->block_size % kQ4Tile) return fail(ZP_ERR_SHAPE, "%s: block_size %d not a multiple of 16", what, D->block_size);
    if (D->h_kv > 256) return fail(ZP_ERR_SHAPE, "%s: h_kv %d > 256", what, D->h_kv);
    if ((long long)D->n_total_blocks * D->block_size > INT32_MAX)
        return fail(ZP_ERR_SHAPE, "%s: %d blocks of %d tokens exceed 32-bit slots", what, D->n_total_blocks, D->block_size);
    return ZP_OK;
}
inline long long q4_layer_bytes(const zp_cache_desc *D, int group) {
    return (long long)D->n_total_blocks * D->h_kv * (D->block_size / kQ4Tile) * q4_tile_bytes(D->head_dim, group);
}

}  // namespace zp
