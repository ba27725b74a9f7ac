// q4_store.cu -- rows quantised into a 4-bit cache, read back from it, and moved
// inside it (format: q4_format.cuh).
//
// Zipage paper §3: the KV cache of a block is written into the block's slots; App. C.6,
// Alg. 4: the kept entries are packed, in order, into the target blocks.  Here the rows are
// held in 4 bits with a step and a lowest value per group of elements.
#include "q4_format.cuh"

namespace zp {
namespace {

// ---------------------------------------------------------------- rows in
// Eight elements of a row per thread (one 16-byte load in bf16, two in fp32): a group of
// 32 is four lanes, its extremes two shuffles away, and a thread's eight codes are one
// 32-bit word, so the 16 lanes of a row of 128 write its 64 bytes side by side.
constexpr int kStoreThreads = 256, kStoreUnroll = 2;

__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <typename T> struct Piece;  // eight elements
template <> struct Piece<__nv_bfloat16> {
    uint4 w;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { w = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = bf2_to_f2(u[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&x)[8]) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(f2_to_bf2(x[0], x[1]), f2_to_bf2(x[2], x[3]), f2_to_bf2(x[4], x[5]),
                                                   f2_to_bf2(x[6], x[7]));
    }
};
template <> struct Piece<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = __ldg(reinterpret_cast<const float4 *>(p));
        b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
        x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    static __device__ __forceinline__ void store(float *p, const float (&x)[8]) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
};

struct StoreArgs {
    const void *k, *v;                       // rows given
    long long token_stride, new_layer_stride;  // elements
    unsigned char *K, *V;
    long long layer_bytes;
    const int32_t *slots;                    // write; append: nullptr
    const int32_t *table, *seq_lens;         // append
    int table_stride;
    int n_tokens, tokens_per_cta;
    int h_kv, b, lg_group, tile;
    int row_pieces;                          // h_kv * d / 8
    unsigned inv_row;                        // ceil(2^32 / row_pieces)
    long long n_slots;
    unsigned *err;
};

// slot of token i (-1: none); the caller's token is within range
template <bool APPEND>
__device__ __forceinline__ long long store_slot(const StoreArgs &a, int i) {
    if constexpr (APPEND) {
        const int L = __ldg(a.seq_lens + i);
        if (L == 0) return -1;  // no token for this sequence in this step
        if (L < 0 || L > (long long)a.table_stride * a.b) {
            record_error(a.err, ZP_ERR_DEVICE, 0x151);
            return -1;
        }
        const int P = L - 1;
        const long long blk = __ldg(a.table + (size_t)i * a.table_stride + P / a.b);
        if (blk < 0 || (blk + 1) * a.b > a.n_slots) {
            record_error(a.err, ZP_ERR_DEVICE, 0x152);
            return -1;
        }
        return blk * a.b + P % a.b;
    } else {
        const long long slot = __ldg(a.slots + i);
        if (slot >= a.n_slots) {
            record_error(a.err, ZP_ERR_DEVICE, 0x150);
            return -1;
        }
        return slot;
    }
}

// tile of (slot, kv head), and the row inside it
__device__ __forceinline__ size_t tile_offset(long long slot, int h, int h_kv, int b, int tile) {
    const int sl = (int)slot, blk = sl / b, in = sl - blk * b;
    return (((size_t)blk * h_kv + h) * (b / kQ4Tile) + in / kQ4Tile) * tile;
}

template <typename T, int D, bool APPEND>
__global__ void __launch_bounds__(kStoreThreads) q4_store_kernel(const StoreArgs a) {
    constexpr int kPieces = D / 8;  // per row
    const T *src = static_cast<const T *>(blockIdx.z ? a.v : a.k) + (long long)blockIdx.y * a.new_layer_stride;
    unsigned char *dst = (blockIdx.z ? a.V : a.K) + (long long)blockIdx.y * a.layer_bytes;
    const int first = blockIdx.x * a.tokens_per_cta;
    const int n = min(a.tokens_per_cta, a.n_tokens - first) * a.row_pieces;
    const int group_lanes = 1 << (a.lg_group - 3);
    for (int base = 0; base < n; base += kStoreThreads * kStoreUnroll) {
        Piece<T> in[kStoreUnroll];
        long long slot[kStoreUnroll];
        int head[kStoreUnroll], piece[kStoreUnroll];
#pragma unroll
        for (int u = 0; u < kStoreUnroll; ++u) {
            const int v = base + u * kStoreThreads + threadIdx.x;
            slot[u] = -1;
            if (v < n) {
                const int i = __umulhi((unsigned)v, a.inv_row);
                const int c = v - i * a.row_pieces;
                in[u].load(src + (long long)(first + i) * a.token_stride + c * 8);
                slot[u] = store_slot<APPEND>(a, first + i);
                head[u] = c / kPieces;
                piece[u] = c % kPieces;
            } else {
                in[u] = Piece<T>{};
            }
        }
#pragma unroll
        for (int u = 0; u < kStoreUnroll; ++u) {
            float x[8];
            in[u].get(x);
            float mn = min_nan(min_nan(min_nan(x[0], x[1]), min_nan(x[2], x[3])), min_nan(min_nan(x[4], x[5]), min_nan(x[6], x[7])));
            float mx = max_nan(max_nan(max_nan(x[0], x[1]), max_nan(x[2], x[3])), max_nan(max_nan(x[4], x[5]), max_nan(x[6], x[7])));
            for (int o = 1; o < group_lanes; o <<= 1) {
                mn = min_nan(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, o));
                mx = max_nan(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
            }
            const uint32_t par = q4_params(mn, mx);
            const float step = __uint_as_float(par << 16), lo = __uint_as_float(par & 0xFFFF0000u);
            const float r = q4_shrunk_reciprocal(step), half = 0.5f * step;
            uint32_t word = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) word |= (q4_code(x[j], lo, step, r, half) & 15u) << (4 * j);
            if (par == kQ4NaN) word = 0;
            if (slot[u] >= 0) {
                const int t = (int)slot[u] % kQ4Tile;
                unsigned char *tile = dst + tile_offset(slot[u], head[u], a.h_kv, a.b, a.tile);
                *reinterpret_cast<uint32_t *>(tile + t * (D / 2) + q4_chunk<D>(t, piece[u] / 4) * 16 + piece[u] % 4 * 4) = word;
                if (piece[u] % group_lanes == 0)
                    reinterpret_cast<uint32_t *>(tile + q4_code_bytes(D))[t * (D >> a.lg_group) + (piece[u] * 8 >> a.lg_group)] = par;
            }
        }
    }
}

// ---------------------------------------------------------------- rows out
constexpr int kReadUnroll = 4;

struct ReadArgs {
    const unsigned char *K, *V;
    long long layer_bytes;
    const int32_t *slots;
    void *k, *v;
    long long token_stride, out_layer_stride;  // elements
    int n_tokens, tokens_per_cta;
    int h_kv, b, lg_group, tile;
    int row_pieces;
    unsigned inv_row;
    long long n_slots;
    unsigned *err;
};

template <typename T, int D>
__global__ void __launch_bounds__(kStoreThreads) q4_read_kernel(const ReadArgs a) {
    constexpr int kPieces = D / 8;
    const unsigned char *src = (blockIdx.z ? a.V : a.K) + (long long)blockIdx.y * a.layer_bytes;
    T *dst = static_cast<T *>(blockIdx.z ? a.v : a.k) + (long long)blockIdx.y * a.out_layer_stride;
    const int first = blockIdx.x * a.tokens_per_cta;
    const int n = min(a.tokens_per_cta, a.n_tokens - first) * a.row_pieces;
    for (int base = 0; base < n; base += kStoreThreads * kReadUnroll) {
        uint32_t word[kReadUnroll], par[kReadUnroll];
        T *to[kReadUnroll];
#pragma unroll
        for (int u = 0; u < kReadUnroll; ++u) {
            const int v = base + u * kStoreThreads + threadIdx.x;
            to[u] = nullptr;
            if (v < n) {
                const int i = __umulhi((unsigned)v, a.inv_row);
                const int c = v - i * a.row_pieces;
                const long long slot = __ldg(a.slots + first + i);
                if (slot >= 0 && slot < a.n_slots) {
                    const int piece = c % kPieces, t = (int)slot % kQ4Tile;
                    const unsigned char *tile = src + tile_offset(slot, c / kPieces, a.h_kv, a.b, a.tile);
                    word[u] = __ldg(reinterpret_cast<const uint32_t *>(tile + t * (D / 2) + q4_chunk<D>(t, piece / 4) * 16 +
                                                                       piece % 4 * 4));
                    par[u] = __ldg(reinterpret_cast<const uint32_t *>(tile + q4_code_bytes(D)) + t * (D >> a.lg_group) +
                                   (piece * 8 >> a.lg_group));
                    to[u] = dst + (long long)(first + i) * a.token_stride + c * 8;
                } else if (slot >= 0) {
                    record_error(a.err, ZP_ERR_DEVICE, 0x153);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kReadUnroll; ++u) {
            if (!to[u]) continue;
            const float step = __uint_as_float(par[u] << 16), lo = __uint_as_float(par[u] & 0xFFFF0000u);
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = fmaf((float)(word[u] >> (4 * j) & 15u), step, lo);
            Piece<T>::store(to[u], x);
        }
    }
}

// ---------------------------------------------------------------- moves
// One CTA per (tensor, kv head, sequence, layer), as in compact.cu: the CTA resolves every
// rank's source and target, then moves up to kMoveChunk ranks at a time: all its row
// pieces (16-byte chunks of codes, 4-byte words of parameters) into registers, a barrier,
// all out.  A chunk reads positions >= its first rank and earlier chunks wrote slots below
// it, and a slot that a source and a target share has the same index in both (the
// target rule): the move is right in place too.
constexpr int kMoveThreads = 1024, kMoveChunk = 2048;

struct MoveArgs {
    unsigned char *K, *V;
    long long layer_bytes;
    float *F;
    long long F_layer_stride;
    const float *S;
    long long S_stride, S_layer_stride;
    const int32_t *S_rows;
    const int32_t *src_table;
    int table_stride;
    const int32_t *dst;
    int target_stride;
    const int32_t *seq_lens, *keep, *k_seq;
    int k, n, h_kv, b, n_total;
    int lg_words, tile;  // log2 of the parameter words of a row
    unsigned *err;
};

template <int D>
__global__ void __launch_bounds__(kMoveThreads, 1) q4_compact_kernel(const MoveArgs a) {
    constexpr int kChunks = D / 32, kPer = kMoveChunk * kChunks / kMoveThreads;  // 16-byte pieces per thread and round
    __shared__ int s_from[kMoveChunk], s_to[kMoveChunk];  // tile * 16 + row, -1: skipped
    const int kvh = blockIdx.x >> 1, tensor = blockIdx.x & 1, s = blockIdx.y, layer = blockIdx.z, tid = threadIdx.x;
    const int32_t *kp = a.keep + (((size_t)layer * a.n + s) * a.h_kv + kvh) * a.k;
    unsigned char *X = (tensor ? a.V : a.K) + layer * a.layer_bytes;
    float *F = a.F && tensor == 0 ? a.F + layer * a.F_layer_stride : nullptr;
    const float *Srow = nullptr;
    int L = __ldg(a.seq_lens + s);
    if (L > (long long)a.table_stride * a.b) L = a.table_stride * a.b;
    if (F) {
        const int row = a.S_rows ? __ldg(a.S_rows + s) : s;
        if (row < 0) {
            if (tid == 0) record_error(a.err, ZP_ERR_DEVICE, 0x156);
            F = nullptr;
        } else {
            Srow = a.S + layer * a.S_layer_stride + ((size_t)row * a.h_kv + kvh) * a.S_stride;
            if (L > a.S_stride) L = (int)a.S_stride;
        }
    }
    const int kk = min(a.k_seq ? min(__ldg(a.k_seq + s), a.k) : a.k, L);
    const int tpb = a.b / kQ4Tile;
    for (int r0 = 0; r0 < kk; r0 += kMoveChunk) {
        const int nr = min(kMoveChunk, kk - r0);
        for (int i = tid; i < nr; i += kMoveThreads) {
            const int r = r0 + i, pos = __ldg(kp + r);
            int from = -1, to = -1, blk = -1;
            if (pos >= 0 && pos < L) blk = __ldg(a.src_table + (size_t)s * a.table_stride + pos / a.b);
            const int target = __ldg(a.dst + (size_t)s * a.target_stride + r / a.b);
            if (blk < 0 || blk >= a.n_total) record_error(a.err, ZP_ERR_DEVICE, 0x154);
            else from = ((blk * a.h_kv + kvh) * tpb + pos % a.b / kQ4Tile) * kQ4Tile + pos % kQ4Tile;
            if (target < 0 || target >= a.n_total) record_error(a.err, ZP_ERR_DEVICE, 0x155);
            else to = ((target * a.h_kv + kvh) * tpb + r % a.b / kQ4Tile) * kQ4Tile + r % kQ4Tile;
            if (to < 0) from = -1;
            s_from[i] = from;
            s_to[i] = to;
            if (F && from >= 0) F[((size_t)target * a.b + r % a.b) * a.h_kv + kvh] = Srow[pos];
        }
        __syncthreads();
        uint4 code[kPer];
        uint32_t par[kMoveChunk * kQ4MaxGroups / kMoveThreads];
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int it = tid + u * kMoveThreads, i = it / kChunks;
            if (i < nr && s_from[i] >= 0) {
                const int t = s_from[i] % kQ4Tile;
                code[u] = *reinterpret_cast<const uint4 *>(X + (size_t)(s_from[i] / kQ4Tile) * a.tile + t * (D / 2) +
                                                           q4_chunk<D>(t, it % kChunks) * 16);
            }
        }
#pragma unroll
        for (int u = 0; u < kMoveChunk * kQ4MaxGroups / kMoveThreads; ++u) {
            const int it = tid + u * kMoveThreads, i = it >> a.lg_words;
            if (i < nr && s_from[i] >= 0)
                par[u] = reinterpret_cast<const uint32_t *>(X + (size_t)(s_from[i] / kQ4Tile) * a.tile + q4_code_bytes(D))
                    [((s_from[i] % kQ4Tile) << a.lg_words) + (it & ((1 << a.lg_words) - 1))];
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int it = tid + u * kMoveThreads, i = it / kChunks;
            if (i < nr && s_from[i] >= 0) {
                const int t = s_to[i] % kQ4Tile;
                *reinterpret_cast<uint4 *>(X + (size_t)(s_to[i] / kQ4Tile) * a.tile + t * (D / 2) +
                                           q4_chunk<D>(t, it % kChunks) * 16) = code[u];
            }
        }
#pragma unroll
        for (int u = 0; u < kMoveChunk * kQ4MaxGroups / kMoveThreads; ++u) {
            const int it = tid + u * kMoveThreads, i = it >> a.lg_words;
            if (i < nr && s_from[i] >= 0)
                reinterpret_cast<uint32_t *>(X + (size_t)(s_to[i] / kQ4Tile) * a.tile + q4_code_bytes(D))
                    [((s_to[i] % kQ4Tile) << a.lg_words) + (it & ((1 << a.lg_words) - 1))] = par[u];
        }
        __syncthreads();  // the next round's loads follow this round's stores
    }
}

int log2_of(int x) {
    int n = 0;
    while ((1 << n) < x) ++n;
    return n;
}

// Tokens per CTA so that one has about `pieces` pieces.
int tokens_per_cta(int row_pieces, int pieces) { return row_pieces >= pieces ? 1 : pieces / row_pieces; }

zp_status check_rows(const zp_cache_desc *D, int group, const char *what, const void *k, const void *v, int64_t token_stride,
                     int64_t rows_layer_stride, int32_t layer_count, const void *K, const void *V, int64_t layer_stride) {
    const int64_t es = elem_bytes(D->dtype), row = (int64_t)D->h_kv * D->head_dim;
    if (layer_count > 65535) return fail(ZP_ERR_SHAPE, "%s: %d layers", what, layer_count);
    if (token_stride < row)
        return fail(ZP_ERR_INVALID_ARG, "%s: token stride %lld below a row of %lld elements", what, (long long)token_stride,
                    (long long)row);
    if (layer_count > 1 && (rows_layer_stride < 0 || layer_stride < q4_layer_bytes(D, group)))
        return fail(ZP_ERR_INVALID_ARG, "%s: layer strides %lld, %lld", what, (long long)rows_layer_stride,
                    (long long)layer_stride);
    const uintptr_t al = (uintptr_t)k | (uintptr_t)v | (uintptr_t)K | (uintptr_t)V;
    if (al % 16 || (token_stride * es) % 16 ||
        (layer_count > 1 && ((rows_layer_stride * es) % 16 || layer_stride % 16)))
        return fail(ZP_ERR_INVALID_ARG, "%s: buffers and strides must be multiples of 16 bytes", what);
    return ZP_OK;
}

template <typename A>
void fill_shape(A &a, const zp_cache_desc *D, int group, int n_tokens, int pieces, const DeviceInfo &dev) {
    a.n_tokens = n_tokens;
    a.h_kv = D->h_kv;
    a.b = D->block_size;
    a.lg_group = log2_of(group);
    a.tile = q4_tile_bytes(D->head_dim, group);
    a.row_pieces = D->h_kv * D->head_dim / 8;
    a.inv_row = (unsigned)((0x100000000ull + a.row_pieces - 1) / a.row_pieces);
    a.tokens_per_cta = tokens_per_cta(a.row_pieces, pieces);
    a.n_slots = (long long)D->n_total_blocks * D->block_size;
    a.err = dev.error_word;
}

template <bool APPEND>
zp_status launch_store(const zp_cache_desc *D, const StoreArgs &a, int layers, const char *what, cudaStream_t st) {
    const dim3 grid((unsigned)((a.n_tokens + (long long)a.tokens_per_cta - 1) / a.tokens_per_cta), (unsigned)layers, 2);
    const bool wide = D->head_dim == 128;
    if (D->dtype == ZP_BF16) {
        if (wide) q4_store_kernel<__nv_bfloat16, 128, APPEND><<<grid, kStoreThreads, 0, st>>>(a);
        else q4_store_kernel<__nv_bfloat16, 64, APPEND><<<grid, kStoreThreads, 0, st>>>(a);
    } else {
        if (wide) q4_store_kernel<float, 128, APPEND><<<grid, kStoreThreads, 0, st>>>(a);
        else q4_store_kernel<float, 64, APPEND><<<grid, kStoreThreads, 0, st>>>(a);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, what);
    return ok();
}

}  // namespace
}  // namespace zp

using namespace zp;

extern "C" size_t zp_q4_tile_bytes(const zp_cache_desc *D, int32_t group) {
    if (check_q4(D, group, "q4_tile_bytes") != ZP_OK) return 0;
    return (size_t)q4_tile_bytes(D->head_dim, group);
}

extern "C" zp_status zp_q4_write_kv(const zp_cache_desc *D, int32_t group, const void *k_new, const void *v_new,
                                    int64_t token_stride, int64_t new_layer_stride, const int32_t *slots,
                                    int32_t n_tokens, void *k_base, void *v_base, int64_t layer_stride,
                                    int32_t layer_count, void *stream) {
    zp_status rc = check_q4(D, group, "q4_write_kv");
    if (rc != ZP_OK) return rc;
    if (n_tokens < 0 || layer_count < 0)
        return fail(ZP_ERR_INVALID_ARG, "q4_write_kv: n_tokens=%d layer_count=%d", n_tokens, layer_count);
    if (n_tokens == 0 || layer_count == 0) return ok();
    if (!k_new || !v_new || !slots || !k_base || !v_base) return fail(ZP_ERR_INVALID_ARG, "q4_write_kv: NULL buffer");
    rc = check_rows(D, group, "q4_write_kv", k_new, v_new, token_stride, new_layer_stride, layer_count, k_base, v_base,
                    layer_stride);
    if (rc != ZP_OK) return rc;
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != ZP_OK) return rc;
    StoreArgs a = {};
    a.k = k_new;
    a.v = v_new;
    a.token_stride = token_stride;
    a.new_layer_stride = layer_count > 1 ? new_layer_stride : 0;
    a.K = static_cast<unsigned char *>(k_base);
    a.V = static_cast<unsigned char *>(v_base);
    a.layer_bytes = layer_count > 1 ? layer_stride : 0;
    a.slots = slots;
    fill_shape(a, D, group, n_tokens, kStoreThreads * kStoreUnroll, dev);
    return launch_store<false>(D, a, layer_count, "q4_write_kv: launch", static_cast<cudaStream_t>(stream));
}

extern "C" zp_status zp_q4_append_kv(const zp_cache_desc *D, int32_t group, const void *k_new, const void *v_new,
                                     void *k_cache, void *v_cache, const int32_t *block_table, int32_t table_stride,
                                     const int32_t *seq_lens, int32_t B, void *stream) {
    zp_status rc = check_q4(D, group, "q4_append_kv");
    if (rc != ZP_OK) return rc;
    if (B < 0 || table_stride < 1)
        return fail(ZP_ERR_INVALID_ARG, "q4_append_kv: B=%d table_stride=%d", B, table_stride);
    if (B == 0) return ok();
    if (!k_new || !v_new || !k_cache || !v_cache || !block_table || !seq_lens)
        return fail(ZP_ERR_INVALID_ARG, "q4_append_kv: NULL buffer");
    const int64_t row = (int64_t)D->h_kv * D->head_dim;
    rc = check_rows(D, group, "q4_append_kv", k_new, v_new, row, 0, 1, k_cache, v_cache, 0);
    if (rc != ZP_OK) return rc;
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != ZP_OK) return rc;
    StoreArgs a = {};
    a.k = k_new;
    a.v = v_new;
    a.token_stride = row;
    a.K = static_cast<unsigned char *>(k_cache);
    a.V = static_cast<unsigned char *>(v_cache);
    a.table = block_table;
    a.table_stride = table_stride;
    a.seq_lens = seq_lens;
    fill_shape(a, D, group, B, kStoreThreads * kStoreUnroll, dev);
    return launch_store<true>(D, a, 1, "q4_append_kv: launch", static_cast<cudaStream_t>(stream));
}

extern "C" zp_status zp_q4_read_kv(const zp_cache_desc *D, int32_t group, const void *k_base, const void *v_base,
                                   int64_t layer_stride, const int32_t *slots, int32_t n_tokens, void *k_out, void *v_out,
                                   int64_t token_stride, int64_t out_layer_stride, int32_t layer_count, void *stream) {
    zp_status rc = check_q4(D, group, "q4_read_kv");
    if (rc != ZP_OK) return rc;
    if (n_tokens < 0 || layer_count < 0)
        return fail(ZP_ERR_INVALID_ARG, "q4_read_kv: n_tokens=%d layer_count=%d", n_tokens, layer_count);
    if (n_tokens == 0 || layer_count == 0) return ok();
    if (!k_base || !v_base || !slots || !k_out || !v_out) return fail(ZP_ERR_INVALID_ARG, "q4_read_kv: NULL buffer");
    rc = check_rows(D, group, "q4_read_kv", k_out, v_out, token_stride, out_layer_stride, layer_count, k_base, v_base,
                    layer_stride);
    if (rc != ZP_OK) return rc;
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != ZP_OK) return rc;
    ReadArgs a = {};
    a.K = static_cast<const unsigned char *>(k_base);
    a.V = static_cast<const unsigned char *>(v_base);
    a.layer_bytes = layer_count > 1 ? layer_stride : 0;
    a.slots = slots;
    a.k = k_out;
    a.v = v_out;
    a.token_stride = token_stride;
    a.out_layer_stride = layer_count > 1 ? out_layer_stride : 0;
    fill_shape(a, D, group, n_tokens, kStoreThreads * kReadUnroll, dev);
    const dim3 grid((unsigned)((n_tokens + (long long)a.tokens_per_cta - 1) / a.tokens_per_cta), (unsigned)layer_count, 2);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool wide = D->head_dim == 128;
    if (D->dtype == ZP_BF16) {
        if (wide) q4_read_kernel<__nv_bfloat16, 128><<<grid, kStoreThreads, 0, st>>>(a);
        else q4_read_kernel<__nv_bfloat16, 64><<<grid, kStoreThreads, 0, st>>>(a);
    } else {
        if (wide) q4_read_kernel<float, 128><<<grid, kStoreThreads, 0, st>>>(a);
        else q4_read_kernel<float, 64><<<grid, kStoreThreads, 0, st>>>(a);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "q4_read_kv: launch");
    return ok();
}

extern "C" zp_status zp_q4_compact_pages(const zp_cache_desc *D, int32_t group, void *k_base, void *v_base,
                                         int64_t layer_stride, int32_t layer_count, float *global_F,
                                         int64_t F_layer_stride, const zp_score_rows *scores, const int32_t *src_table,
                                         int32_t table_stride, const int32_t *dst_targets, int32_t target_stride,
                                         const int32_t *seq_lens, const int32_t *keep_idx, int32_t k,
                                         const int32_t *k_seq, int32_t n, void *stream) {
    zp_status rc = check_q4(D, group, "q4_compact");
    if (rc != ZP_OK) return rc;
    if (n < 0 || k < 0 || layer_count < 0 || table_stride < 1 || target_stride < 1)
        return fail(ZP_ERR_INVALID_ARG, "q4_compact: n=%d k=%d layer_count=%d table_stride=%d target_stride=%d", n, k,
                    layer_count, table_stride, target_stride);
    if (n == 0 || k == 0 || layer_count == 0) return ok();
    if (!k_base || !v_base || !src_table || !dst_targets || !seq_lens || !keep_idx)
        return fail(ZP_ERR_INVALID_ARG, "q4_compact: NULL buffer");
    if (global_F && (!scores || !scores->data || scores->stride < 1))
        return fail(ZP_ERR_INVALID_ARG, "q4_compact: global_F needs the score rows");
    if ((long long)target_stride * D->block_size < k)
        return fail(ZP_ERR_CAPACITY, "q4_compact: %d target blocks hold fewer than k=%d rows", target_stride, k);
    if (n > 65535 || layer_count > 65535) return fail(ZP_ERR_SHAPE, "q4_compact: n=%d layer_count=%d", n, layer_count);
    if ((long long)D->n_total_blocks * D->block_size * D->h_kv > INT32_MAX)
        return fail(ZP_ERR_SHAPE, "q4_compact: %d blocks of %d tokens and %d heads exceed 32-bit rows", D->n_total_blocks,
                    D->block_size, D->h_kv);
    if (layer_count > 1 && layer_stride < q4_layer_bytes(D, group))
        return fail(ZP_ERR_INVALID_ARG, "q4_compact: layer_stride %lld < one layer", (long long)layer_stride);
    if (((uintptr_t)k_base | (uintptr_t)v_base) % 16 || (layer_count > 1 && layer_stride % 16))
        return fail(ZP_ERR_INVALID_ARG, "q4_compact: caches and layer_stride must be multiples of 16 bytes");
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != ZP_OK) return rc;
    MoveArgs a = {};
    a.K = static_cast<unsigned char *>(k_base);
    a.V = static_cast<unsigned char *>(v_base);
    a.layer_bytes = layer_count > 1 ? layer_stride : 0;
    a.F = global_F;
    a.F_layer_stride = layer_count > 1 ? F_layer_stride : 0;
    a.S = global_F ? scores->data : nullptr;
    a.S_stride = global_F ? scores->stride : 1;
    a.S_layer_stride = global_F && layer_count > 1 ? scores->layer_stride : 0;
    a.S_rows = global_F ? scores->rows : nullptr;
    a.src_table = src_table;
    a.table_stride = table_stride;
    a.dst = dst_targets;
    a.target_stride = target_stride;
    a.seq_lens = seq_lens;
    a.keep = keep_idx;
    a.k_seq = k_seq;
    a.k = k;
    a.n = n;
    a.h_kv = D->h_kv;
    a.b = D->block_size;
    a.n_total = D->n_total_blocks;
    a.lg_words = log2_of(D->head_dim / group);
    a.tile = q4_tile_bytes(D->head_dim, group);
    a.err = dev.error_word;
    const dim3 grid(2 * D->h_kv, n, layer_count);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (D->head_dim == 128) q4_compact_kernel<128><<<grid, kMoveThreads, 0, st>>>(a);
    else q4_compact_kernel<64><<<grid, kMoveThreads, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "q4_compact: launch");
    return ok();
}
