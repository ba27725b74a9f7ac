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
constexpr uint32_t kQ4NaN = 0x7FC07FC0u;  // step and lo of a group that holds anything not finite

__host__ __device__ constexpr int q4_code_bytes(int d) { return kQ4Tile * d / 2; }
__host__ __device__ constexpr int q4_tile_bytes(int d, int group) { return q4_code_bytes(d) + kQ4Tile * 4 * (d / group); }

// The same value, which the compiler knows only from here on.  What is loaded from an address that comes from
// it stays behind the waits and barriers before: they are volatile as this is, and a load without a memory
// clobber (a read-only or cached one) is otherwise free to pass them.  Costs no instruction.
template <typename T>
__device__ __forceinline__ T *from_here(T *p) {
    asm volatile("" : "+l"(p));
    return p;
}
__device__ __forceinline__ int from_here(int x) {
    asm volatile("" : "+r"(x));
    return x;
}

template <int D>
__host__ __device__ __forceinline__ int q4_chunk(int t, int c) {
    return D == 128 ? (c ^ ((t >> 1) & 3)) : (c ^ ((t >> 2) & 1));
}

// bf16 bits of the largest bf16 value not above x (x not NaN).
__device__ __forceinline__ uint32_t bf16_below(float x) {
    const uint32_t u = __float_as_uint(x);
    return ((u & 0xFFFFu) && (u >> 31) ? u + 0x10000u : u) >> 16;
}

// The word (step, lo) of a group whose smallest and largest element are mn and mx
// (NaN if one of its elements is): lo is the bf16 value at or below mn, the step the
// smallest bf16 value of which fifteen reach from lo to mx, so that no element is further than
// half a step, and what x - lo is rounded by, from its code's value.  For bf16 elements lo is mn
// itself.  The step is at least 2^-126 (its reciprocal is finite).
__device__ __forceinline__ uint32_t q4_params(float mn, float mx) {
    const uint32_t lo = bf16_below(mn);
    const float flo = __uint_as_float(lo << 16), spread = mx - flo;
    // a fifteenth, a little too large (0x3D88888B is 2.8e-7 above 1/15), cut to bf16: the answer or the value below it
    uint32_t s = __float_as_uint(spread * __uint_as_float(0x3D88888Bu)) & 0xFFFF0000u;
    if (15.f * __uint_as_float(s) < spread) s += 0x10000u;  // (15 s has 12 bits)
    const float step = fmaxf(__uint_as_float(s), __uint_as_float(0x00800000u));
    const bool finite = fabsf(flo) < INFINITY && spread < INFINITY;  // (a NaN compares false)
    return finite ? (__float_as_uint(step) >> 16) | (lo << 16) : kQ4NaN;
}

// ---- codes: of x in a group with (step, lo), floor((x - lo) / step + 1/2), the quotient not
// rounded.  r is a reciprocal of the step too small by 2^-20 or so, so that k, (x - lo) * r
// rounded, is the code or one less; (k + 1/2) * step is exact (13 bits) and tells which.
__device__ __forceinline__ float q4_small_reciprocal(float step) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(step));  // off by 2^-23 at most
    return r * (1.f - 9.5367431640625e-7f);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(*reinterpret_cast<unsigned long long *>(&a)), "l"(*reinterpret_cast<unsigned long long *>(&b)));
    return *reinterpret_cast<float2 *>(&r);
}
__device__ __forceinline__ float at_least(float a, float b) {  // 1 where a >= b, else 0
    float r;
    asm("set.ge.f32.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Codes of two elements, as floats.
__device__ __forceinline__ float2 q4_code2(float2 x, float lo, float step, float r, float half) {
    const float2 d = add2(x, both(-lo));
    const float2 k = add2(ffma2(d, both(r), both(12582912.f)), both(-12582912.f));  // 1.5 * 2^23: rounds to a whole number
    const float2 edge = ffma2(k, both(step), both(half));
    return add2(k, make_float2(at_least(d.x, edge.x), at_least(d.y, edge.y)));
}
// Eight whole numbers of 0 to 15, of two words, as the nibbles of those (four make a
// number below 2^16, which 2^23 shows as the low bits).
__device__ __forceinline__ uint2 q4_join(const float2 (&k)[8]) {
    float2 x[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        x[h] = add2(ffma2(k[4 * h + 3], both(4096.f), ffma2(k[4 * h + 2], both(256.f), ffma2(k[4 * h + 1], both(16.f), k[4 * h]))),
                    both(8388608.f));
    return make_uint2(__byte_perm(__float_as_uint(x[0].x), __float_as_uint(x[1].x), 0x5410),
                      __byte_perm(__float_as_uint(x[0].y), __float_as_uint(x[1].y), 0x5410));
}

// Code j of a word as a float.  Nibbles 0 to 4 stay where they are: under the exponent of 2^(23 - 4j) the bits
// from 4j on count ones.
__device__ __forceinline__ float q4_code_at(uint32_t w, int j) {
    if (j > 4) w >>= 20, j -= 5;
    return __uint_as_float((w & 15u << (4 * j)) | (uint32_t)(150 - 4 * j) << 23) - (float)(1 << (23 - 4 * j));
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
