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
// Sixteen elements of a row per thread (32 bytes in bf16, 64 in fp32): a group of 32 is two
// lanes, its extremes one shuffle away, its parameters are worked out for 16 elements at a
// time, and a thread's codes are 8 bytes, so the 8 lanes of a row of 128 write its 64 bytes
// side by side.  A thread keeps its place in the row and walks over tokens.
// Bound: for many rows the instructions, about 14 per element and lane, issued in three quarters of all cycles:
// 64k tokens of 8 heads of 128 in bf16, 352 MB, take 67 us (5.2 TB/s, 0.78 of a plain copy's rate); for few
// the launch (512 tokens 2.6 us).  One row at a time per thread: with two the registers cost what the second
// load in flight gains (64k tokens 1 us more), and 512 tokens take longer.
constexpr int kStoreThreads = 256, kPiece = 16;

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
__device__ __forceinline__ uint32_t min_nan2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max_nan2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// 32 bytes; in one access where the rows are 32-byte aligned
__device__ __forceinline__ void load32(uint32_t (&w)[8], const void *p, bool wide) {
    if (wide) {
        asm("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
            : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
            : "l"(p));
    } else {
        const uint4 x = __ldg(static_cast<const uint4 *>(p)), y = __ldg(static_cast<const uint4 *>(p) + 1);
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w, w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
    }
}
__device__ __forceinline__ void store32(void *p, const uint32_t (&w)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        static_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

template <typename T> struct Piece;  // sixteen elements
template <> struct Piece<__nv_bfloat16> {
    uint32_t w[8];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p, bool wide) { load32(w, p, wide); }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 0;
    }
    __device__ __forceinline__ float get(int i) const {
        return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    }
    __device__ __forceinline__ void extremes(float &mn, float &mx) const {
        uint32_t a = w[0], b = w[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) a = min_nan2(a, w[i]), b = max_nan2(b, w[i]);
        const float2 x = bf2_to_f2(a), y = bf2_to_f2(b);
        mn = min_nan(x.x, x.y);
        mx = max_nan(y.x, y.y);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&x)[16], bool wide) {
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = f2_to_bf2(x[2 * i], x[2 * i + 1]);
        store32(p, o, wide);
    }
};
template <> struct Piece<float> {
    uint32_t a[8], b[8];
    __device__ __forceinline__ void load(const float *p, bool wide) {
        load32(a, p, wide);
        load32(b, p + 8, wide);
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = b[i] = 0;
    }
    __device__ __forceinline__ float get(int i) const { return __uint_as_float(i < 8 ? a[i & 7] : b[i & 7]); }
    __device__ __forceinline__ void extremes(float &mn, float &mx) const {
        mn = mx = get(0);
#pragma unroll
        for (int i = 1; i < 16; ++i) mn = min_nan(mn, get(i)), mx = max_nan(mx, get(i));
    }
    static __device__ __forceinline__ void store(float *p, const float (&x)[16], bool wide) {
        uint32_t o[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(x[8 * h + i]);
            store32(p + 8 * h, o, wide);
        }
    }
};

// What the calls that go over rows share.  A CTA has lanes_n threads for each of `at_once`
// tokens at a time (a thread for every kPiece elements of a row, or fewer where a row has more
// than kStoreThreads of them) and takes tokens_per_cta in all.
struct RowArgs {
    int n_tokens, tokens_per_cta, at_once, lanes_n;
    int h_kv, lg_group, tile;
    int row_pieces;                   // h_kv * d / kPiece
    int tpb;                          // tiles per block and kv head
    unsigned inv_lanes, inv_tpb;      // reciprocals, rounded up, of 2^32 (0: the divisor is 1)
    int n_slots;
    bool wide;                        // rows aligned to 32 bytes
    unsigned *err;
};

// Byte offset of the tile of a slot from that of its kv head's first tile: the tiles of a head and block lie
// tpb apart times h_kv, so ((slot / b) * h_kv * tpb + slot % b / 16) * tile, in 32-bit factors.
__device__ __forceinline__ size_t tile_offset(const RowArgs &a, int slot) {
    const unsigned t = (unsigned)slot / kQ4Tile;  // below 2^27; the reciprocal is exact as far as that
    unsigned m = t;                               // the first tile of the block
    if (a.inv_tpb) {
        m = __umulhi(t, a.inv_tpb) * a.tpb;
        if (m > t) m -= a.tpb;  // (rounded up: one too many at most)
    }
    return (size_t)m * (unsigned)((a.h_kv - 1) * a.tile) + (size_t)t * (unsigned)a.tile;
}

struct StoreArgs : RowArgs {
    const void *k, *v;                         // rows given
    long long token_stride, new_layer_stride;  // elements
    unsigned char *K, *V;
    long long layer_bytes;
    const int32_t *slots;             // write; append: nullptr
    const int32_t *table, *seq_lens;  // append
    int table_stride;
};

// slot of token i, -1: none
template <bool APPEND>
__device__ __forceinline__ int store_slot(const StoreArgs &a, int i) {
    if constexpr (APPEND) {
        const int L = __ldg(from_here(a.seq_lens) + i), b = a.tpb * kQ4Tile;
        if (L == 0) return -1;  // no token for this sequence in this step
        if (L < 0 || L > (long long)a.table_stride * b) {
            record_error(a.err, ZP_ERR_DEVICE, 0x151);
            return -1;
        }
        const int P = L - 1;
        const long long blk = __ldg(from_here(a.table) + (size_t)i * a.table_stride + P / b);
        if (blk < 0 || (blk + 1) * b > a.n_slots) {
            record_error(a.err, ZP_ERR_DEVICE, 0x152);
            return -1;
        }
        return (int)(blk * b + P % b);
    } else {
        const int slot = __ldg(from_here(a.slots) + i);
        if (slot >= a.n_slots) {
            record_error(a.err, ZP_ERR_DEVICE, 0x150);
            return -1;
        }
        return slot;
    }
}

template <typename T, int D, bool APPEND, int U>
__global__ void __launch_bounds__(kStoreThreads) q4_store_kernel(const StoreArgs a) {
    constexpr int kPieces = D / kPiece;  // per row of a head
    const T *src = static_cast<const T *>(blockIdx.z ? a.v : a.k) + (long long)blockIdx.y * a.new_layer_stride;
    unsigned char *dst = (blockIdx.z ? a.V : a.K) + (long long)blockIdx.y * a.layer_bytes;
    const int tok = a.inv_lanes ? (int)__umulhi(threadIdx.x, a.inv_lanes) : (int)threadIdx.x;
    const int first = blockIdx.x * a.tokens_per_cta + tok, last = min(a.n_tokens, ((int)blockIdx.x + 1) * a.tokens_per_cta);
    const int group_lanes = 1 << (a.lg_group - 4), lg_row = 2 + (D == 128 ? 7 : 6) - a.lg_group;  // log2 of a row's parameter bytes
    const long long step_rows = a.at_once * a.token_stride;
    pdl_wait();
    // (every thread goes as often round as the first: the shuffles are the whole warp's)
    for (int c0 = 0; c0 < a.row_pieces; c0 += a.lanes_n) {
        const int c = from_here((int)(c0 + threadIdx.x - tok * a.lanes_n));  // (the rows' addresses come from it)
        const int head = c / kPieces, piece = c % kPieces;
        const bool works = tok < a.at_once && c < a.row_pieces;
        const T *from = src + (long long)first * a.token_stride + c * kPiece;
        unsigned char *base = dst + (size_t)head * a.tpb * a.tile;
        const int par_at = q4_code_bytes(D) + (piece * kPiece >> a.lg_group) * 4;
        for (int i0 = first; i0 - tok < last; i0 += U * a.at_once) {
            Piece<T> in[U];
            int slot[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * a.at_once;
                slot[u] = -1;
                if (works && i < last) {
                    in[u].load(from, a.wide);
                    slot[u] = store_slot<APPEND>(a, i);
                } else {
                    in[u].clear();
                }
                from += step_rows;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float mn, mx;
                in[u].extremes(mn, mx);
                for (int o = 1; o < group_lanes; o <<= 1) {
                    mn = min_nan(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, o));
                    mx = max_nan(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
                }
                const uint32_t par = q4_params(mn, mx);
                const float step = __uint_as_float(par << 16), lo = __uint_as_float(par & 0xFFFF0000u);
                const float r = q4_small_reciprocal(step), half = 0.5f * step;
                float2 k[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) k[j] = q4_code2(make_float2(in[u].get(j), in[u].get(j + 8)), lo, step, r, half);
                uint2 word = q4_join(k);
                if (par == kQ4NaN) word = make_uint2(0, 0);
                if (slot[u] < 0) continue;
                const int t = slot[u] % kQ4Tile;
                unsigned char *tile = base + tile_offset(a, slot[u]);
                *reinterpret_cast<uint2 *>(tile + t * (D / 2) + q4_chunk<D>(t, piece / 2) * 16 + piece % 2 * 8) = word;
                if (piece % group_lanes == 0) *reinterpret_cast<uint32_t *>(tile + (t << lg_row) + par_at) = par;
            }
        }
    }
}

// ---------------------------------------------------------------- rows out
// The same threads and walk, the other way, two rows at a time: 64k tokens of 8 heads of 128 into
// bf16 take 58 us (6.0 TB/s, 0.90 of a plain copy's rate: bound by memory), 1,024 tokens 2.8; with
// four rows 1 us less and 0.7 more, with one 4 more and the same.
struct ReadArgs : RowArgs {
    const unsigned char *K, *V;
    long long layer_bytes;
    const int32_t *slots;
    void *k, *v;
    long long token_stride, out_layer_stride;  // elements
};

template <typename T, int D, int U>
__global__ void __launch_bounds__(kStoreThreads) q4_read_kernel(const ReadArgs a) {
    constexpr int kPieces = D / kPiece;
    const unsigned char *src = (blockIdx.z ? a.V : a.K) + (long long)blockIdx.y * a.layer_bytes;
    T *dst = static_cast<T *>(blockIdx.z ? a.v : a.k) + (long long)blockIdx.y * a.out_layer_stride;
    const int tok = a.inv_lanes ? (int)__umulhi(threadIdx.x, a.inv_lanes) : (int)threadIdx.x;
    pdl_wait();
    if (tok >= a.at_once) return;
    const int first = blockIdx.x * a.tokens_per_cta + tok, last = min(a.n_tokens, ((int)blockIdx.x + 1) * a.tokens_per_cta);
    const int lg_row = 2 + (D == 128 ? 7 : 6) - a.lg_group;  // log2 of a row's parameter bytes
    const long long step_rows = a.at_once * a.token_stride;
    for (int c = threadIdx.x - tok * a.lanes_n; c < a.row_pieces; c += a.lanes_n) {
        const int head = c / kPieces, piece = c % kPieces;
        T *to = dst + (long long)first * a.token_stride + c * kPiece;
        const unsigned char *base = from_here(src) + (size_t)head * a.tpb * a.tile;
        const int par_at = q4_code_bytes(D) + (piece * kPiece >> a.lg_group) * 4;
        for (int i0 = first; i0 < last; i0 += U * a.at_once) {
            uint2 word[U];
            uint32_t par[U];
            int slot[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * a.at_once;
                slot[u] = i < last ? __ldg(from_here(a.slots) + i) : -1;
                if (slot[u] >= a.n_slots) {
                    record_error(a.err, ZP_ERR_DEVICE, 0x153);
                    slot[u] = -1;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (slot[u] < 0) continue;
                const int t = slot[u] % kQ4Tile;
                const unsigned char *tile = base + tile_offset(a, slot[u]);
                word[u] = __ldg(reinterpret_cast<const uint2 *>(tile + t * (D / 2) + q4_chunk<D>(t, piece / 2) * 16 + piece % 2 * 8));
                par[u] = __ldg(reinterpret_cast<const uint32_t *>(tile + (t << lg_row) + par_at));
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (slot[u] >= 0) {
                    const float step = __uint_as_float(par[u] << 16), lo = __uint_as_float(par[u] & 0xFFFF0000u);
                    float x[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) x[j] = fmaf(q4_code_at(j < 8 ? word[u].x : word[u].y, j & 7), step, lo);
                    Piece<T>::store(to, x, a.wide);
                }
                to += step_rows;
            }
        }
    }
}

// ---------------------------------------------------------------- moves
// One CTA per (tensor, kv head, sequence, layer) moves its ranks in rounds of kMoveRanks (a thread
// each) through a ring in shared memory: asynchronous copies in, kMoveStages - 1 rounds ahead,
// plain stores out.  Round i is stored once all of its copies have arrived.  Its stores go to slots
// below the ranks of later rounds, whose sources are at or above those ranks, and a slot that a
// source and a target share has the same index in both (the target rule): later rounds may be read
// ahead of earlier stores, and the move is right in place too.  A row in flight costs no registers
// that way, and the look-ups (position, then block) run a round or two ahead of the copies.
// Bound: memory, where a row has 64 bytes of codes and 16 of parameters far from them.  16 sequences, 4080 of 32k
// tokens each, 8 heads of 128: 56 us for 84 MB of rows, for which 232 MB are read and 49 MB written (5.0 TB/s);
// 7 sequences of 2032 rows 12.5 us, a chain of five latencies (length, position, block, row, store).
// Rows that went through registers, a round's loads before its stores, took 104 us where the ring took 58.
constexpr int kMoveStages = 4;

__device__ __forceinline__ void copy_async(void *to, const void *from, int bytes) {  // 4, 8 or 16
    const uint32_t at = smem_u32(to);
    if (bytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
    else if (bytes == 8) asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(at), "l"(from) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(at), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

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

// A stage: codes [ranks][d/2], parameters [ranks][words], F values [ranks], 1 where the rank moves [ranks].
__host__ __device__ constexpr int move_stage_bytes(int ranks, int d, int words) { return ranks * (d / 2 + 4 * words + 8); }

template <int D, int kMoveRanks>
__global__ void __launch_bounds__(kMoveRanks) q4_compact_kernel(const MoveArgs a) {
    constexpr int kChunks = D / 32, kRows = 32 / kChunks;  // rows that a warp copies at a time
    extern __shared__ __align__(16) unsigned char smem[];
    const int kvh = blockIdx.x >> 1, tensor = blockIdx.x & 1, s = blockIdx.y, layer = blockIdx.z;
    const int tid = threadIdx.x, lane = tid & 31, warp0 = tid & ~31;
    const int words = 1 << a.lg_words, stage_bytes = move_stage_bytes(kMoveRanks, D, words), tpb = a.b / kQ4Tile;
    const int32_t *kp = a.keep + (((size_t)layer * a.n + s) * a.h_kv + kvh) * a.k;
    const int32_t *table = a.src_table + (size_t)s * a.table_stride, *dst = a.dst + (size_t)s * a.target_stride;
    unsigned char *X = (tensor ? a.V : a.K) + layer * a.layer_bytes;
    float *F = a.F && tensor == 0 ? a.F + layer * a.F_layer_stride : nullptr;
    const float *Srow = nullptr;
    pdl_wait();
    kp = from_here(kp), table = from_here(table), dst = from_here(dst);
    int pos_b = tid < a.k ? __ldg(kp + tid) : -1, pos_c = tid + kMoveRanks < a.k ? __ldg(kp + tid + kMoveRanks) : -1;
    int L = (int)min((long long)__ldg(from_here(a.seq_lens) + s), (long long)a.table_stride * a.b);
    if (F) {
        const int row = a.S_rows ? __ldg(from_here(a.S_rows) + s) : s;
        if (row < 0) {
            if (tid == 0) record_error(a.err, ZP_ERR_DEVICE, 0x156);
            F = nullptr;
        } else {
            Srow = a.S + layer * a.S_layer_stride + ((size_t)row * a.h_kv + kvh) * a.S_stride;
            if (L > a.S_stride) L = (int)a.S_stride;
        }
    }
    const int kk = min(a.k_seq ? min(__ldg(from_here(a.k_seq) + s), a.k) : a.k, L);
    const int rounds = (kk + kMoveRanks - 1) / kMoveRanks;
    auto block_of = [&](int pos) { return pos >= 0 && pos < L ? __ldg(table + pos / a.b) : -1; };
    int pos = pos_b, blk = block_of(pos_b);  // of the next round to copy
    pos_b = pos_c;                           // of the one behind it
    // the copies of round i: lane l looks rank r up, kChunks lanes copy a row's codes
    auto copy = [&](int i) {
        if (i < rounds) {
            unsigned char *stage = smem + (i % kMoveStages) * stage_bytes;
            unsigned char *par = stage + kMoveRanks * (D / 2);
            float *f = reinterpret_cast<float *>(par + kMoveRanks * 4 * words);
            int *moves = reinterpret_cast<int *>(f + kMoveRanks);
            const int r = i * kMoveRanks + tid;
            int from = -1;  // tile * 16 + row
            if (r < kk) {
                if (blk < 0 || blk >= a.n_total) record_error(a.err, ZP_ERR_DEVICE, 0x154);
                else from = ((blk * a.h_kv + kvh) * tpb + pos % a.b / kQ4Tile) * kQ4Tile + pos % kQ4Tile;
            }
            moves[tid] = from >= 0;
            if (from >= 0) {
                copy_async(par + tid * 4 * words, X + (size_t)(from / kQ4Tile) * a.tile + q4_code_bytes(D) + from % kQ4Tile * 4 * words,
                           4 * words);
                if (F) copy_async(f + tid, Srow + pos, 4);
            }
#pragma unroll
            for (int u = 0; u < kChunks; ++u) {
                const int row = u * kRows + lane / kChunks, x = __shfl_sync(0xFFFFFFFFu, from, row), c = lane % kChunks;
                if (x >= 0)
                    copy_async(stage + (warp0 + row) * (D / 2) + c * 16,
                               X + (size_t)(x / kQ4Tile) * a.tile + x % kQ4Tile * (D / 2) + q4_chunk<D>(x % kQ4Tile, c) * 16, 16);
            }
            pos = pos_b;
            blk = block_of(pos_b);
            const int far = r + 2 * kMoveRanks;
            pos_b = far < a.k ? __ldg(kp + far) : -1;
        }
        copies_commit();
    };
    for (int i = 0; i < kMoveStages - 1; ++i) copy(i);
    for (int i = 0; i < rounds; ++i) {
        copies_wait<kMoveStages - 2>();
        __syncthreads();  // round i is here, and round i - 1 has been stored: its stage is free
        copy(i + kMoveStages - 1);
        const unsigned char *stage = smem + (i % kMoveStages) * stage_bytes;
        const unsigned char *par = stage + kMoveRanks * (D / 2);
        const float *f = reinterpret_cast<const float *>(par + kMoveRanks * 4 * words);
        const int *moves = reinterpret_cast<const int *>(f + kMoveRanks);
        const int r = i * kMoveRanks + tid;
        int to = -1;
        if (r < kk) {
            const int target = __ldg(dst + r / a.b);
            if (target < 0 || target >= a.n_total) {
                record_error(a.err, ZP_ERR_DEVICE, 0x155);
            } else if (moves[tid]) {
                to = ((target * a.h_kv + kvh) * tpb + r % a.b / kQ4Tile) * kQ4Tile + r % kQ4Tile;
                unsigned char *at = X + (size_t)(to / kQ4Tile) * a.tile + q4_code_bytes(D) + to % kQ4Tile * 4 * words;
                if (words == 4) *reinterpret_cast<uint4 *>(at) = reinterpret_cast<const uint4 *>(par)[tid];
                else if (words == 2) *reinterpret_cast<uint2 *>(at) = reinterpret_cast<const uint2 *>(par)[tid];
                else *reinterpret_cast<uint32_t *>(at) = reinterpret_cast<const uint32_t *>(par)[tid];
                if (F) F[((size_t)target * a.b + r % a.b) * a.h_kv + kvh] = f[tid];
            }
        }
#pragma unroll
        for (int u = 0; u < kChunks; ++u) {
            const int row = u * kRows + lane / kChunks, x = __shfl_sync(0xFFFFFFFFu, to, row), c = lane % kChunks;
            if (x >= 0)
                *reinterpret_cast<uint4 *>(X + (size_t)(x / kQ4Tile) * a.tile + x % kQ4Tile * (D / 2) + q4_chunk<D>(x % kQ4Tile, c) * 16) =
                    *reinterpret_cast<const uint4 *>(stage + (warp0 + row) * (D / 2) + c * 16);
        }
    }
}

int log2_of(int x) {
    int n = 0;
    while ((1 << n) < x) ++n;
    return n;
}

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

// Do rows of k and v, of any tokens and layers, have a byte in common?  (Tokens are a row apart at least.)
bool rows_meet(const zp_cache_desc *D, const void *k, const void *v, int64_t n, int64_t token_stride, int64_t layer_stride,
               int64_t layers) {
    const int64_t es = elem_bytes(D->dtype), row = (int64_t)D->h_kv * D->head_dim * es, ts = token_stride * es;
    const int64_t ls = layers > 1 ? layer_stride * es : 0, apart = (int64_t)((uintptr_t)v - (uintptr_t)k);
    // two lines of n rows, one `by` bytes behind the other: the multiples of ts next to `by` decide
    auto meet = [&](int64_t by) {
        if (by < 0) by = -by;
        const int64_t i = by / ts;
        return (i < n && by - i * ts < row) || (i + 1 < n && (i + 1) * ts - by < row);
    };
    if (ls < (n - 1) * ts + row)  // (else every layer is behind the one before)
        for (int64_t l = 1; l < layers; ++l)
            if (meet(l * ls)) return true;
    const int64_t all = (layers - 1) * ls + (n - 1) * ts + row;
    if (apart < all && -apart < all)
        for (int64_t l = 1 - layers; l < layers; ++l)
            if (meet(apart + l * ls)) return true;
    return false;
}

// Bits that the addresses of rows have in common with their strides.
uintptr_t row_alignment(const zp_cache_desc *D, const void *k, const void *v, int64_t token_stride, int64_t layer_stride) {
    const int64_t es = elem_bytes(D->dtype);
    return (uintptr_t)k | (uintptr_t)v | (uintptr_t)(token_stride * es) | (uintptr_t)(layer_stride * es);
}

unsigned reciprocal(int x) { return x == 1 ? 0 : (unsigned)((0x100000000ull + x - 1) / x); }

// The split of n_tokens rows (of `layers` layers, keys and values) over CTAs whose threads
// take U tokens at a time.
void fill_rows(RowArgs &a, const zp_cache_desc *D, int group, int n_tokens, int layers, int U, uintptr_t aligned,
               const DeviceInfo &dev) {
    a.n_tokens = n_tokens;
    a.row_pieces = D->h_kv * D->head_dim / kPiece;
    a.lanes_n = a.row_pieces < kStoreThreads ? a.row_pieces : kStoreThreads;
    a.at_once = kStoreThreads / a.lanes_n;
    // Where there are far more CTAs than the SMs hold, each goes round up to 8 times (what a thread works out
    // once is then spread over more rows) as long as several CTAs per SM and place remain to even the end out.
    const long long ctas = ((long long)n_tokens + a.at_once * U - 1) / (a.at_once * U) * layers * 2;
    const long long rounds = ctas / (dev.sm_count * 20);
    a.tokens_per_cta = a.at_once * U * (int)(rounds < 1 ? 1 : rounds > 8 ? 8 : rounds);
    a.h_kv = D->h_kv;
    a.lg_group = log2_of(group);
    a.tile = q4_tile_bytes(D->head_dim, group);
    a.tpb = D->block_size / kQ4Tile;
    a.inv_lanes = reciprocal(a.lanes_n);
    a.inv_tpb = reciprocal(a.tpb);
    a.n_slots = D->n_total_blocks * D->block_size;
    a.wide = aligned % 32 == 0;
    a.err = dev.error_word;
}
dim3 row_grid(const RowArgs &a, int layers) {
    return dim3((unsigned)((a.n_tokens + (long long)a.tokens_per_cta - 1) / a.tokens_per_cta), (unsigned)layers, 2);
}

constexpr int kStoreUnroll = 1, kReadUnroll = 2;

template <bool APPEND>
zp_status launch_store(const zp_cache_desc *D, const StoreArgs &a, int layers, const char *what, cudaStream_t st) {
    const bool wide = D->head_dim == 128;
    const auto kernel = D->dtype == ZP_BF16
                            ? (wide ? q4_store_kernel<__nv_bfloat16, 128, APPEND, kStoreUnroll> : q4_store_kernel<__nv_bfloat16, 64, APPEND, kStoreUnroll>)
                            : (wide ? q4_store_kernel<float, 128, APPEND, kStoreUnroll> : q4_store_kernel<float, 64, APPEND, kStoreUnroll>);
    const cudaError_t e = launch_dependent(kernel, row_grid(a, layers), dim3(kStoreThreads), 0, st, a);
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
    if (n_tokens > 1 << 30) return fail(ZP_ERR_SHAPE, "q4_write_kv: %d tokens", n_tokens);
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
    fill_rows(a, D, group, n_tokens, layer_count, kStoreUnroll, row_alignment(D, k_new, v_new, token_stride, a.new_layer_stride), dev);
    return launch_store<false>(D, a, layer_count, "q4_write_kv: launch", static_cast<cudaStream_t>(stream));
}

extern "C" zp_status zp_q4_append_kv(const zp_cache_desc *D, int32_t group, const void *k_new, const void *v_new,
                                     void *k_cache, void *v_cache, const int32_t *block_table, int32_t table_stride,
                                     const int32_t *seq_lens, int32_t B, void *stream) {
    zp_status rc = check_q4(D, group, "q4_append_kv");
    if (rc != ZP_OK) return rc;
    if (B < 0 || table_stride < 1)
        return fail(ZP_ERR_INVALID_ARG, "q4_append_kv: B=%d table_stride=%d", B, table_stride);
    if (B > 1 << 30) return fail(ZP_ERR_SHAPE, "q4_append_kv: %d tokens", B);
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
    fill_rows(a, D, group, B, 1, kStoreUnroll, row_alignment(D, k_new, v_new, row, 0), dev);
    return launch_store<true>(D, a, 1, "q4_append_kv: launch", static_cast<cudaStream_t>(stream));
}

extern "C" zp_status zp_q4_read_kv(const zp_cache_desc *D, int32_t group, const void *k_base, const void *v_base,
                                   int64_t layer_stride, const int32_t *slots, int32_t n_tokens, void *k_out, void *v_out,
                                   int64_t token_stride, int64_t out_layer_stride, int32_t layer_count, void *stream) {
    zp_status rc = check_q4(D, group, "q4_read_kv");
    if (rc != ZP_OK) return rc;
    if (n_tokens < 0 || layer_count < 0)
        return fail(ZP_ERR_INVALID_ARG, "q4_read_kv: n_tokens=%d layer_count=%d", n_tokens, layer_count);
    if (n_tokens > 1 << 30) return fail(ZP_ERR_SHAPE, "q4_read_kv: %d tokens", n_tokens);
    if (n_tokens == 0 || layer_count == 0) return ok();
    if (!k_base || !v_base || !slots || !k_out || !v_out) return fail(ZP_ERR_INVALID_ARG, "q4_read_kv: NULL buffer");
    rc = check_rows(D, group, "q4_read_kv", k_out, v_out, token_stride, out_layer_stride, layer_count, k_base, v_base,
                    layer_stride);
    if (rc != ZP_OK) return rc;
    if (rows_meet(D, k_out, v_out, n_tokens, token_stride, out_layer_stride, layer_count))
        return fail(ZP_ERR_INVALID_ARG, "q4_read_kv: rows of the output lie on one another (token stride %lld, layer stride %lld)",
                    (long long)token_stride, (long long)out_layer_stride);
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
    fill_rows(a, D, group, n_tokens, layer_count, kReadUnroll, row_alignment(D, k_out, v_out, token_stride, a.out_layer_stride), dev);
    const bool wide = D->head_dim == 128;
    const auto kernel = D->dtype == ZP_BF16
                            ? (wide ? q4_read_kernel<__nv_bfloat16, 128, kReadUnroll> : q4_read_kernel<__nv_bfloat16, 64, kReadUnroll>)
                            : (wide ? q4_read_kernel<float, 128, kReadUnroll> : q4_read_kernel<float, 64, kReadUnroll>);
    const cudaError_t e = launch_dependent(kernel, row_grid(a, layer_count), dim3(kStoreThreads), 0, static_cast<cudaStream_t>(stream), a);
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
    if (n > 65535 || layer_count > 65535 || k > 1 << 30)
        return fail(ZP_ERR_SHAPE, "q4_compact: n=%d layer_count=%d k=%d", n, layer_count, k);
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
    // Rounds of 512 ranks where every CTA has an SM of its own (7 sequences of 2032 ranks 12.5 us,
    // with 256 16.5), of 256 and two or more CTAs per SM where there are more (16 of 4080: 56 us, 60).
    const dim3 grid(2 * D->h_kv, n, layer_count);
    const bool few = (long long)grid.x * grid.y * grid.z <= dev.sm_count, wide = D->head_dim == 128;
    const int ranks = few ? 512 : 256;
    const auto kernel = wide ? (few ? q4_compact_kernel<128, 512> : q4_compact_kernel<128, 256>)
                             : (few ? q4_compact_kernel<64, 512> : q4_compact_kernel<64, 256>);
    const size_t smem = (size_t)kMoveStages * move_stage_bytes(ranks, D->head_dim, D->head_dim / group);
    rc = set_max_dynamic_smem(reinterpret_cast<const void *>(kernel), smem, "q4_compact: shared-memory attribute");
    if (rc != ZP_OK) return rc;
    const cudaError_t e = launch_dependent(kernel, grid, dim3(ranks), smem, static_cast<cudaStream_t>(stream), a);
    if (e != cudaSuccess) return cuda_fail(e, "q4_compact: launch");
    return ok();
}
