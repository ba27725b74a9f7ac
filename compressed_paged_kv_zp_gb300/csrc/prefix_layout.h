// prefix_layout.h -- places in a query tile of the tensor-core prefix kernels
// (plain arithmetic, so that the host can check it too).
#pragma once

#ifdef __CUDACC__
#define ZP_LAYOUT_FN __host__ __device__ constexpr
#else
#define ZP_LAYOUT_FN constexpr
#endif

namespace zp {

// Byte offset of 16-byte chunk `chunk` of row `row`: a tile is made of 64-element
// halves `half` bytes apart, a row of a half is 128 bytes, its chunks exchanged by
// the 128-byte swizzle of the copies and descriptors.
//
// Two users, whose places must coincide warp by warp, since the warps of a stream
// are not ordered with one another between them: a warp's query rows, and the rows
// of its records, which pass through the same tile once the products that read it
// are complete (chunk c of record row r then lies where chunk c of query row r
// did).  A warp owns rows [32 w, 32 w + 32) in both, and so touches no byte of
// another's.
ZP_LAYOUT_FN int pt_chunk(int row, int chunk, int half) {
    return (chunk >> 3) * half + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

// fp32 columns of a record that pass through the tile at a time: what fits in the
// bytes of a row's D bf16 queries.
ZP_LAYOUT_FN int pt_record_cols(int D) { return D / 2; }

}  // namespace zp
