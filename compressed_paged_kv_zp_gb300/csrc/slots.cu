// slots.cu -- block tables and slot maps built on the GPU from request
// lengths, and the keys and values of many tokens stored through a slot map.
//
// zp_build_slots: sequence s grows from o_s to n_s tokens.  Its touched columns
// are floor(o_s/b) .. ceil(n_s/b)-1 (none when n_s = o_s); those at or beyond
// ceil(o_s/b) whose table entry is negative are missing and take the fresh
// blocks in (sequence, column) order.  Token t of [o_s, n_s) is output
// cu[s] + (t - o_s), its slot table[t/b]*b + t%b.
//
// One launch: every CTA scans the lengths of all sequences (B <= 4096, 32 KB)
// into shared memory, takes an equal contiguous share of the touched columns,
// needs the number of missing entries before its share, and then deals blocks
// and writes slots for its own columns, whose tokens are contiguous in the
// output.  A CTA counts what lies before it from the table entries of the touched
// columns (B of them in a decode step, new tokens / b in a prefill).  Beyond a few
// entries per thread a cluster of 8 CTAs counts together and exchanges the counts
// in distributed shared memory.  Latency bound: the redundant scan and count cost
// less than a second launch (512 sequences of a token each 6.0 us, 16 prompts of 32k
// tokens, half a million slots, 12.6 us).  In place (table_out = block_table) there is one
// cluster, since the counts read entries that other clusters would write (in place, every
// block placed already: 7.8 and 48.6 us).
#include <cooperative_groups.h>

#include "zp_common.cuh"

namespace zp {
namespace {

constexpr int kSlotThreads = 512;
constexpr int kSlotMaxB = 4096;
constexpr int kSlotCluster = 8;  // CTAs of a cluster

struct SlotArgs {
    const int32_t *table;
    int32_t *table_out;
    int stride;
    const int32_t *old_lens, *new_lens;
    int B, b, n_total;
    const int32_t *fresh;
    int n_fresh;
    int32_t *slots, *positions;
    int max_tokens;
    int32_t *cu, *n_used;
    unsigned *err;
};

// Exclusive scan over the CTA (blockDim = kSlotThreads); *total gets the sum.
__device__ __forceinline__ int block_scan(int x, int *warp_sums, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int v = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += y;
    }
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int w = lane < kSlotThreads / 32 ? warp_sums[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, w, o);
            if (lane >= o) w += y;
        }
        if (lane < kSlotThreads / 32) warp_sums[lane] = w;
    }
    __syncthreads();
    const int before = warp ? warp_sums[warp - 1] : 0;
    *total = warp_sums[kSlotThreads / 32 - 1];
    __syncthreads();
    return before + v - x;
}

// Lengths of sequence s; a bad pair counts as no growth.
__device__ __forceinline__ int2 slot_lens(const SlotArgs &a, int s, bool record) {
    int o = a.old_lens[s], n = a.new_lens[s];
    if (o < 0 || n < o || n > a.stride * a.b) {
        if (record) record_error(a.err, ZP_ERR_DEVICE, 0x120);
        o = n = 0;
    }
    return make_int2(o, n);
}

// last s in [0, B) with start[s] <= x[k], for N values at once (their loads
// overlap); top: the largest power of two below B (0 for one sequence)
template <int N>
__device__ __forceinline__ void find_seq(const int *start, int B, int top, const int (&x)[N], int (&s)[N]) {
#pragma unroll
    for (int k = 0; k < N; ++k) s[k] = 0;
    for (int step = top; step; step >>= 1) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int t = s[k] + step;
            if (t < B && start[t] <= x[k]) s[k] = t;
        }
    }
}

template <bool kCluster>
__global__ void __launch_bounds__(kSlotThreads) build_slots_kernel(const SlotArgs a) {
    extern __shared__ int slot_smem[];
    int *ccol = slot_smem;              // [B+1] touched columns before s
    int *ctok = ccol + a.B + 1;         // [B+1] new tokens before s
    int *old_s = ctok + a.B + 1;        // [B] old length
    int *col_s = old_s + a.B;           // [B] first touched column * 2 + (it holds old tokens: never missing)
    __shared__ int warp_sums[kSlotThreads / 32];
    __shared__ int counts[2];  // missing entries this CTA counted before its cluster, and in its own share
    __shared__ int blk_s[kSlotThreads], tok_s[kSlotThreads], n_s[kSlotThreads], pos_s[kSlotThreads];
    const int tid = threadIdx.x;
    const bool lead = blockIdx.x == 0;
    int cols = 0, toks = 0;  // totals so far
    for (int base = 0; base < a.B; base += kSlotThreads) {
        const int s = base + tid;
        int c = 0, t = 0;
        if (s < a.B) {
            const int2 l = slot_lens(a, s, lead);
            t = l.y - l.x;
            c = t ? (l.y + a.b - 1) / a.b - l.x / a.b : 0;
            old_s[s] = l.x;
            const int c0 = l.x / a.b;
            col_s[s] = 2 * c0 + (l.x > c0 * a.b ? 1 : 0);
        }
        int ct, tt;
        const int ce = block_scan(c, warp_sums, &ct), te = block_scan(t, warp_sums, &tt);
        if (s < a.B) {
            ccol[s] = cols + ce;
            ctok[s] = toks + te;
            if (lead) a.cu[s] = toks + te;
        }
        cols += ct;
        toks += tt;
    }
    if (tid == 0) {
        ccol[a.B] = cols;
        ctok[a.B] = toks;
        if (lead) a.cu[a.B] = toks;
    }
    __syncthreads();
    const int G = gridDim.x;
    const int x0 = (int)((long long)cols * blockIdx.x / G), x1 = (int)((long long)cols * (blockIdx.x + 1) / G);

    int top = 1;
    while (2 * top < a.B) top *= 2;
    if (a.B < 2) top = 0;
    // Missing entries (no block yet, and not the column of old tokens) of the
    // touched columns [xb, xe): those of group `which` of every `every`.
    constexpr int kAhead = 8;  // table entries in flight per thread
    auto count = [&](int xb, int xe, int which, int every) {
        int found = 0;
        for (int g0 = xb + which * kSlotThreads * kAhead; g0 < xe; g0 += every * kSlotThreads * kAhead) {
            int e[kAhead];
#pragma unroll
            for (int k0 = 0; k0 < kAhead; k0 += 2) {  // (two searches at a time; none beyond the range)
                e[k0] = e[k0 + 1] = 0;
                if (g0 + k0 * kSlotThreads >= xe) continue;
                const int x[2] = {g0 + k0 * kSlotThreads + tid, g0 + (k0 + 1) * kSlotThreads + tid};
                int s[2];
                find_seq<2>(ccol, a.B, top, x, s);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int i = x[k] - ccol[s[k]], c = col_s[s[k]];
                    if (x[k] < xe && !(i == 0 && (c & 1))) e[k0 + k] = a.table[(size_t)s[k] * a.stride + (c >> 1) + i];
                }
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) found += e[k] < 0 ? 1 : 0;
        }
        return found;
    };
    int before;
    if constexpr (kCluster) {
        auto cluster = cooperative_groups::this_cluster();
        const int rank = (int)cluster.block_rank(), c_first = blockIdx.x - rank;
        const int xc = (int)((long long)cols * c_first / G);  // the cluster's first column
        int n_before, n_own;
        block_scan(count(0, xc, rank, kSlotCluster), warp_sums, &n_before);
        block_scan(count(x0, x1, 0, 1), warp_sums, &n_own);
        if (tid == 0) {
            counts[0] = n_before;
            counts[1] = n_own;
        }
        cluster.sync();
        int n = 0;
        if (tid < kSlotCluster) {
            const int *c = cluster.map_shared_rank(counts, tid);
            n = c[0] + (tid < rank ? c[1] : 0);
        }
        block_scan(n, warp_sums, &before);
        cluster.sync();  // the counts have been read (and, in place, every table entry that the counts need)
    } else {
        block_scan(count(0, x0, 0, 1), warp_sums, &before);
    }
    if (a.table_out != a.table) {
        // copy of the table; the touched columns are written by their owners
        const int n_table = a.B * a.stride;  // (below 2^31 by the limits)
        for (long long i = (long long)blockIdx.x * kSlotThreads + tid; i < n_table; i += (long long)G * kSlotThreads) {
            const int s = (int)((unsigned)i / (unsigned)a.stride), c = (int)i - s * a.stride;
            const int n_cols = ccol[s + 1] - ccol[s], c0 = col_s[s] >> 1;
            if (n_cols == 0 || c < c0 || c >= c0 + n_cols) a.table_out[i] = a.table[i];
        }
    }
    for (int base = x0; base < x1; base += kSlotThreads) {
        const int x = base + tid;
        int s = 0, c = 0, miss = 0, entry = 0;
        if (x < x1) {
            const int xs[1] = {x};
            int found[1];
            find_seq<1>(ccol, a.B, top, xs, found);
            s = found[0];
            c = (col_s[s] >> 1) + (x - ccol[s]);
            entry = a.table[(size_t)s * a.stride + c];
            miss = entry < 0 && !(x == ccol[s] && (col_s[s] & 1)) ? 1 : 0;
        }
        int total;
        const int rank = before + block_scan(miss, warp_sums, &total);
        before += total;
        int cnt = 0;
        if (x < x1) {
            int blk;
            if (miss) {
                blk = rank < a.n_fresh ? a.fresh[rank] : -1;
                if (rank >= a.n_fresh) record_error(a.err, ZP_ERR_DEVICE, 0x121);
            } else {
                blk = entry;
            }
            a.table_out[(size_t)s * a.stride + c] = blk;
            if ((blk < 0 || blk >= a.n_total) && !(miss && rank >= a.n_fresh))
                record_error(a.err, ZP_ERR_DEVICE, 0x122);
            const int o = old_s[s], n = o + ctok[s + 1] - ctok[s];
            const int t0 = max(o, c * a.b);
            cnt = min(n, (c + 1) * a.b) - t0;
            blk_s[tid] = blk >= 0 && blk < a.n_total ? blk : -1;
            tok_s[tid] = ctok[s] + t0 - o;
            pos_s[tid] = t0;
        }
        n_s[tid] = cnt;
        __syncthreads();
        // 16 lanes per column: the tokens of consecutive columns are consecutive outputs
        const int n_here = min(kSlotThreads, x1 - base);
        for (int k = tid / 16; k < n_here; k += kSlotThreads / 16) {
            const int blk = blk_s[k], i0 = tok_s[k], t0 = pos_s[k];
            for (int j = tid % 16; j < n_s[k]; j += 16) {
                const int i = i0 + j, t = t0 + j;
                if (i >= a.max_tokens) {
                    record_error(a.err, ZP_ERR_DEVICE, 0x123);
                    break;
                }
                a.slots[i] = blk < 0 ? -1 : blk * a.b + t % a.b;
                if (a.positions) a.positions[i] = t;
            }
        }
        __syncthreads();
    }
    if (a.n_used && tid == 0 && blockIdx.x == G - 1) *a.n_used = before;
    // padding behind the last token
    for (long long i = toks + (long long)blockIdx.x * kSlotThreads + tid; i < a.max_tokens;
         i += (long long)G * kSlotThreads) {
        a.slots[i] = -1;
        if (a.positions) a.positions[i] = -1;
    }
}

// ---------------------------------------------------------------------------
// zp_write_kv: row i (one token, every kv head) of layer l goes to slot
// slots[i] of that layer.  A copy, bound by HBM: a thread has kWriteUnroll vectors of
// 16 bytes in flight, a CTA's vectors are consecutive.  16k tokens of 4 layers, 8 heads
// of 128 in bf16, 528 MB read and written: 76 us, 6.9 TB/s (with 8 vectors 78, with one
// 86).  Few tokens are bound by the latency of slot and row: 509 tokens of 2 fp32 heads of
// 64 2.1 us (with 8 vectors, so a quarter of the CTAs, 4.4).
struct WriteArgs {
    const uint4 *k, *v;
    long long token_vec, new_layer_vec;  // strides of k, v in 16-byte vectors
    uint4 *K, *V;
    long long layer_vec;
    const int32_t *slots;
    int n_tokens, row_vec;
    long long n_slots;
    unsigned *err;
};

constexpr int kWriteThreads = 256, kWriteUnroll = 2;

__global__ void __launch_bounds__(kWriteThreads) write_kv_kernel(const WriteArgs a) {
    const uint4 *src = (blockIdx.z ? a.v : a.k) + (long long)blockIdx.y * a.new_layer_vec;
    uint4 *dst = (blockIdx.z ? a.V : a.K) + (long long)blockIdx.y * a.layer_vec;
    const long long n = (long long)a.n_tokens * a.row_vec;
    const long long v0 = (long long)blockIdx.x * (kWriteThreads * kWriteUnroll) + threadIdx.x;
    uint4 x[kWriteUnroll];
    long long to[kWriteUnroll];
#pragma unroll
    for (int u = 0; u < kWriteUnroll; ++u) {
        const long long v = v0 + u * kWriteThreads;
        to[u] = -1;
        if (v < n) {
            const int i = (int)(v / a.row_vec);
            const int c = (int)(v - (long long)i * a.row_vec);
            const long long slot = __ldg(a.slots + i);
            if (slot >= 0 && slot < a.n_slots) {
                to[u] = slot * a.row_vec + c;
                x[u] = __ldg(src + i * a.token_vec + c);
            } else if (slot >= 0) {
                record_error(a.err, ZP_ERR_DEVICE, 0x130);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < kWriteUnroll; ++u)
        if (to[u] >= 0) dst[to[u]] = x[u];
}

}  // namespace
}  // namespace zp

using namespace zp;

extern "C" zp_status zp_build_slots(const zp_cache_desc *D, const int32_t *block_table, int32_t *table_out,
                                    int32_t table_stride, const int32_t *old_lens, const int32_t *new_lens, int32_t B,
                                    const int32_t *fresh, int32_t n_fresh, int32_t *slots, int32_t *positions,
                                    int32_t max_tokens, int32_t *cu_tokens, int32_t *n_used, void *stream) {
    zp_status rc = check_desc(D);
    if (rc != ZP_OK) return rc;
    if (B < 0 || table_stride < 1 || n_fresh < 0 || max_tokens < 0)
        return fail(ZP_ERR_INVALID_ARG, "build_slots: B=%d table_stride=%d n_fresh=%d max_tokens=%d", B, table_stride,
                    n_fresh, max_tokens);
    if (!cu_tokens || (B > 0 && (!block_table || !table_out || !old_lens || !new_lens)) || (n_fresh > 0 && !fresh) ||
        (max_tokens > 0 && !slots))
        return fail(ZP_ERR_INVALID_ARG, "build_slots: NULL buffer");
    const uintptr_t t_in = (uintptr_t)block_table, t_out = (uintptr_t)table_out;
    const uintptr_t t_bytes = (uintptr_t)B * table_stride * 4;
    if (t_in != t_out && t_in < t_out + t_bytes && t_out < t_in + t_bytes)
        return fail(ZP_ERR_INVALID_ARG, "build_slots: table_out overlaps block_table without being it");
    if (B > kSlotMaxB) return fail(ZP_ERR_SHAPE, "build_slots: B %d > %d", B, kSlotMaxB);
    if ((long long)D->n_total_blocks * D->block_size > INT32_MAX ||
        (long long)B * table_stride * D->block_size > INT32_MAX)
        return fail(ZP_ERR_SHAPE, "build_slots: %d blocks of %d tokens, or B=%d rows of %d blocks, exceed 32-bit slots",
                    D->n_total_blocks, D->block_size, B, table_stride);
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != ZP_OK) return rc;
    SlotArgs a = {block_table, table_out, table_stride, old_lens, new_lens, B, D->block_size, D->n_total_blocks, fresh,
                  n_fresh, slots, positions, max_tokens, cu_tokens, n_used, dev.error_word};
    // the columns that new tokens can touch, at most: per sequence one, and one
    // per b tokens.  Up to 4096 of them a CTA counts alone (512 sequences, one
    // token each: 6.0 us; in clusters 10.5), beyond that in clusters (16 prompts of
    // 32k tokens: 12.6 us; alone 22.5).
    const long long most = (long long)B + max_tokens / D->block_size;
    const bool in_place = table_out == block_table, clusters = in_place || most > 4096;
    const size_t smem = (size_t)(4 * B + 2) * 4;
    const auto kernel = clusters ? build_slots_kernel<true> : build_slots_kernel<false>;
    rc = set_max_dynamic_smem(reinterpret_cast<const void *>(kernel), smem, "build_slots: shared-memory attribute");
    if (rc != ZP_OK) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(in_place ? kSlotCluster : (unsigned)align_up(dev.sm_count, kSlotCluster));
    cfg.blockDim = dim3(kSlotThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kSlotCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = clusters ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    if (e != cudaSuccess) return cuda_fail(e, "build_slots: launch");
    return ok();
}

extern "C" zp_status zp_write_kv(const zp_cache_desc *D, const void *k_new, const void *v_new, int64_t token_stride,
                                 int64_t new_layer_stride, const int32_t *slots, int32_t n_tokens, void *k_base,
                                 void *v_base, int64_t layer_stride, int32_t layer_count, void *stream) {
    zp_status rc = check_desc(D);
    if (rc != ZP_OK) return rc;
    if (n_tokens < 0 || layer_count < 0)
        return fail(ZP_ERR_INVALID_ARG, "write_kv: n_tokens=%d layer_count=%d", n_tokens, layer_count);
    if (n_tokens == 0 || layer_count == 0) return ok();
    if (!k_new || !v_new || !slots || !k_base || !v_base) return fail(ZP_ERR_INVALID_ARG, "write_kv: NULL buffer");
    if (layer_count > 65535) return fail(ZP_ERR_SHAPE, "write_kv: %d layers", layer_count);
    const int64_t es = elem_bytes(D->dtype), row = (int64_t)D->h_kv * D->head_dim;
    if (token_stride < row) return fail(ZP_ERR_INVALID_ARG, "write_kv: token stride %lld below a row of %lld elements",
                                        (long long)token_stride, (long long)row);
    if (layer_count > 1 && (new_layer_stride < 0 || layer_stride < (int64_t)D->n_total_blocks * D->block_size * row))
        return fail(ZP_ERR_INVALID_ARG, "write_kv: layer strides %lld, %lld", (long long)new_layer_stride,
                    (long long)layer_stride);
    const uintptr_t al = (uintptr_t)k_new | (uintptr_t)v_new | (uintptr_t)k_base | (uintptr_t)v_base;
    if (al % 16 || (token_stride * es) % 16 || (layer_count > 1 && ((new_layer_stride * es) % 16 || (layer_stride * es) % 16)))
        return fail(ZP_ERR_INVALID_ARG, "write_kv: buffers and strides must be multiples of 16 bytes");
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != ZP_OK) return rc;
    WriteArgs a;
    a.k = static_cast<const uint4 *>(k_new);
    a.v = static_cast<const uint4 *>(v_new);
    a.token_vec = token_stride * es / 16;
    a.new_layer_vec = layer_count > 1 ? new_layer_stride * es / 16 : 0;
    a.K = static_cast<uint4 *>(k_base);
    a.V = static_cast<uint4 *>(v_base);
    a.layer_vec = layer_count > 1 ? layer_stride * es / 16 : 0;
    a.slots = slots;
    a.n_tokens = n_tokens;
    a.row_vec = (int)(row * es / 16);
    a.n_slots = (long long)D->n_total_blocks * D->block_size;
    a.err = dev.error_word;
    const long long n = (long long)n_tokens * a.row_vec, per = kWriteThreads * kWriteUnroll;
    const long long gx = (n + per - 1) / per;
    if (gx > INT32_MAX) return fail(ZP_ERR_SHAPE, "write_kv: %d rows of %d vectors", n_tokens, a.row_vec);
    write_kv_kernel<<<dim3((unsigned)gx, (unsigned)layer_count, 2), kWriteThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "write_kv: launch");
    return ok();
}
