// zp_internal.h -- declarations shared by the translation units of libzp.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "zp.h"

namespace zp {

// Host: record a message for zp_last_error() and return the status.
zp_status fail(zp_status s, const char *fmt, ...);
zp_status cuda_fail(cudaError_t e, const char *where);
zp_status ok();

// Host: properties of the current device (cached per device).
struct DeviceInfo {
    int device;
    int sm_count;
    int smem_optin;  // max dynamic shared memory per block
    unsigned *error_word;  // device address of the status word
};
zp_status device_info(DeviceInfo *out);

// Host: raise the dynamic shared-memory limit of kernel `func` on the current
// device to at least `bytes` (one call per kernel, device and larger size;
// safe from several host threads).  A failure
// returns ZP_ERR_CUDA with `what` in the message.
zp_status set_max_dynamic_smem(const void *func, size_t bytes, const char *what);

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

inline int elem_bytes(int dtype) { return dtype == ZP_BF16 ? 2 : (dtype == ZP_F32 ? 4 : 0); }

zp_status check_desc(const zp_cache_desc *D);

// Host: a 3-D tiled tensor map of bf16 elements with the 128-byte swizzle
// (tensor maps for the TMA loads of tcgen05 operands).  dims innermost first;
// strides (bytes) of dims 1 and 2; box innermost first (box[0] * 2 <= 128).
// Encoded through the driver entry point (no link against libcuda).
zp_status encode_tmap_bf16_3d(void *map /* CUtensorMap */, const void *base, const uint64_t dims[3],
                              const uint64_t strides[2], const uint32_t box[3], const char *what);

// The same of any rank from 2 to 5 (rank - 1 strides).
zp_status encode_tmap_bf16(void *map, int rank, const void *base, const uint64_t *dims, const uint64_t *strides,
                           const uint32_t *box, const char *what);

// All-pairs key redundancy of one layer (redundancy.cu): rho [n][h_kv][Lmax]
// receives the row sums of the thresholded cosine matrix of every sequence and
// kv head (overwritten).  Lengths are clamped to Lcap.
struct AllPairsArgs {
    const void *k;  // paged keys of the layer
    int dtype;      // ZP_BF16 or ZP_F32
    const int32_t *table;
    int table_stride;
    const int32_t *seq_lens;
    int n, h_kv, d, b, n_total, Lmax, Lcap;
    float p;
    float *rho;
    void *workspace;  // all_pairs_workspace_size bytes
};
size_t all_pairs_workspace_size(int n, int h_kv, int d, int Lmax);
zp_status launch_all_pairs(const AllPairsArgs &a, cudaStream_t st);

// Host: launch as a programmatic dependent of the kernel before it on the stream
// (the kernel calls pdl_wait() before it reads what that one writes).
template <typename... P, typename... A>
inline cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// The decode of the tokens behind the prefixes (arguments checked as for
// zp_paged_decode_attn; the workspace is the decode's), its records joined with
// those of the prefix kernel (pfx) into the outputs.  With score_accum it leaves,
// and tells pfx, what the score of all tokens needs: the final statistics of every
// entry, the logits of the entries on a window step and the units they lie in.
struct PfxArgs;
zp_status decode_after_prefix(const zp_cache_desc *D, const void *q, const void *k_cache, const void *v_cache,
                              const int32_t *block_table, int32_t table_stride, const int32_t *seq_lens, int32_t B,
                              void *out, float *score_accum, const int32_t *score_rows, int32_t n_score_rows,
                              int32_t window, PfxArgs &pfx, void *workspace, size_t workspace_bytes, void *stream);

}  // namespace zp
