// q4_decode.cu -- paged GQA decode attention over a 4-bit cache, with the window score.
//
// For every sequence s and query head h (Zipage paper §3, §6; the score is App. C.2's):
//     out[s][h] = sum_{t<L_s} softmax_t(q[s][h] . k_t / sqrt(d)) v_t,
// k_t and v_t the values that the cache's codes stand for (q4_format.cuh).
//
// Work unit = two tiles (32 tokens) of one kv head.  The units of all (sequence, kv head)
// pairs are laid one after another and every warp takes an equal contiguous range, so
// ragged lengths cannot unbalance the grid.  A warp copies the tiles of its range to a ring of
// its own in shared memory (bulk copies, one mbarrier per stage) and runs an online softmax in
// base 2 over them.  A pair that lies in one warp's range is written out by it.  Of a pair cut
// between warps each keeps a record (reference, sums, accumulator) in shared memory; at the end
// the CTA joins them and writes the pair out, or one record of it to the workspace where it
// goes on in other CTAs.  q4_finish_kernel joins those (at most one pair per CTA boundary) and,
// on window steps, turns the logits that the attention left (log2 units) into probabilities
// with the final sums, takes the maximum over the q heads and adds 1/w of it to the score.
// With few pairs a pair's units are cut between the CTAs of a cluster instead, and nothing else is
// launched (pick_cluster).
//
// Bound: a 4-bit row of 128 elements is 80 bytes, for which every q head asks 128 multiplications:
// with many tokens the issue of instructions (390 of a warp for 16 tokens, nearly half of them on
// the half-rate integer pipe) and the memory are near one another, below that the time before the
// first copy and after the last product.  Of keys and values, 32 q and 8 kv heads of 128, groups of
// 32, with a copy's rate as 1:
//     512 sequences of 1k to 4k tokens   324 us  5.2 TB/s  0.78
//      64 of 4k at most                   51      4.1      0.62   (first copy at 4.3 us, last product at 43)
//     256 of 4k at most, scored          172      4.0      0.60   (logits written and read besides)
//       1 of 32k                          20.7    2.0      0.31   (3.4 units per warp: latencies)
//       4 of 2k                           12.6                    (latencies: lengths, table, tiles, join)
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <math.h>

#include <map>
#include <mutex>
#include <utility>

#include "q4_format.cuh"

namespace zp {
namespace {

constexpr int kQ4MaxB = 4096;
constexpr int kUnit = 2 * kQ4Tile;  // tokens of a unit
constexpr int kMaxStages = 4;       // units a warp has in flight, at most

struct Q4Args {
    const void *q;
    const unsigned char *k, *v;
    void *out;
    const int32_t *table;
    int table_stride;
    const int32_t *seq_lens;
    int B, h_q, h_kv, G, b, n_total;
    int tile, tpb;  // bytes of a tile, tiles of a block and kv head
    unsigned inv_tpb, inv_ranges;  // reciprocals (div_by) of tpb and of the CTAs * warps that share a split
    float qscale;   // log2(e) / sqrt(d)
    int want_score, window;
    float *score;
    long long score_stride;
    const int32_t *score_rows;
    int n_score_rows;
    int *prefix;    // [B+1] units before each sequence (of one kv head)
    float2 *stats;  // [B][h_q] reference and log2(sum) of the pairs that one CTA saw whole
    float *rec;     // [2 * CTAs + warps][G * (d + 4)]: per head (reference, sum for the output, sum, 0), then accumulators
    float *logits;  // [units][32][G]
    int grid, warps, stages;  // CTAs of the attention kernel, warps of one, units in a warp's ring
    int pair_units;           // units that the table has room for (cluster: the logits of a pair)
    int cluster;              // 0: all pairs are one line, cut evenly; else the CTAs (a cluster) of every pair
    bool heads_here;          // records of pairs that began before a warp's range: in shared memory
    unsigned *err;
};

// ---------------------------------------------------------------- the split
// n / d for n below 2^31, inv = 2^32 / d rounded up (d > 1) or 0 (d = 1): the product is one
// too large at most.
__device__ __forceinline__ int div_by(int n, int d, unsigned inv) {
    if (!inv) return n;
    const int q = (int)__umulhi((unsigned)n, inv);
    return q - (q * d > n);
}

struct Split {
    int U, W;           // units, ranges (no more than units: none is empty)
    int per_cta, ctas;  // ranges of a CTA (its first warps take one each), CTAs that have some
    int quot, rest;     // U / W, U % W
    unsigned inv_W;
    // the first unit of range g: floor(g U / W)  (W is below 2^15: g * rest below 2^30)
    __device__ __forceinline__ int start(int g) const { return g * quot + div_by(g * rest, W, inv_W); }
    __device__ __forceinline__ int cta_start(int c) const { return start(c * per_cta); }
    // the CTA whose ranges hold unit x: the largest range g with start(g) <= x is its
    __device__ __forceinline__ int cta_of(int x) const { return (int)(((x + 1ll) * W - 1) / U) / per_cta; }
};

__device__ __forceinline__ Split make_split(const Q4Args &a, int units, int grid) {
    Split p;
    p.U = units;
    if (p.U >= grid * a.warps) {
        p.per_cta = a.warps;
        p.ctas = grid;
        p.inv_W = a.inv_ranges;
    } else {
        const int want = (int)(((unsigned)p.U + grid - 1) / (unsigned)grid);
        p.per_cta = want < 1 ? 1 : want;
        const int most = p.U / p.per_cta;
        p.ctas = most < grid ? most : grid;
        const int W = p.per_cta * p.ctas;
        p.inv_W = W <= 1 ? 0u : 0xFFFFFFFFu / (unsigned)W + 1;
    }
    p.W = p.per_cta * p.ctas;
    p.quot = div_by(p.U, p.W, p.inv_W);
    p.rest = p.U - p.quot * p.W;
    return p;
}

// A length as it is taken, the nearer bound where it lies outside [0, table_stride * b].
__device__ __forceinline__ int checked_len(const Q4Args &a, int L) {
    const long long cap = (long long)a.table_stride * a.b;
    if (L < 0 || L > cap) {
        record_error(a.err, ZP_ERR_DEVICE, 0x158);
        return L < 0 ? 0 : (int)cap;
    }
    return L;
}
__device__ __forceinline__ int units_of(int L) { return (int)(((long long)L + kUnit - 1) / kUnit); }
__device__ __forceinline__ int q4_len(const Q4Args &a, int s) { return checked_len(a, __ldg(from_here(a.seq_lens) + s)); }

// prefix[s] = units of the sequences before s; blockDim.x threads, a multiple of 32.
__device__ void unit_prefix(const Q4Args &a, int *prefix, int *warp_sum) {
    const int per = (a.B + blockDim.x - 1) / blockDim.x;
    const int s0 = min((int)threadIdx.x * per, a.B), s1 = min(s0 + per, a.B);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int mine = 0;
    for (int s = s0; s < s1; ++s) {
        const int n = units_of(q4_len(a, s));
        prefix[s] = n;
        mine += n;
    }
    int x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int before = x - mine;
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    for (int s = s0; s < s1; ++s) {
        const int n = prefix[s];
        prefix[s] = before;
        before += n;
    }
    if (threadIdx.x == blockDim.x - 1) prefix[a.B] = before;
    __syncthreads();
}

// A place in the sequence of units.
struct Cursor {
    int s, h, u, n;  // unit u of the n of (sequence s, kv head h)
    __device__ __forceinline__ void seek(const int *prefix, int B, int h_kv, int x) {
        int lo = 0, hi = B - 1;
        while (lo < hi) {  // the last s with prefix[s] * h_kv <= x (it has units)
            const int mid = (lo + hi + 1) >> 1;
            if (prefix[mid] * h_kv <= x) lo = mid;
            else hi = mid - 1;
        }
        s = lo;
        n = prefix[s + 1] - prefix[s];
        const int in = x - prefix[s] * h_kv;
        h = in / n;
        u = in - h * n;
    }
    // unit x of the pair that the CTA's cluster has
    __device__ __forceinline__ void at(const Q4Args &a, int x) {
        const int pair = (int)blockIdx.x / a.cluster;
        s = pair / a.h_kv;
        h = pair - s * a.h_kv;
        u = x;
        n = units_of(q4_len(a, s));
    }
    __device__ __forceinline__ void next(const int *prefix, int B, int h_kv) {
        if (++u < n) return;
        u = 0;
        if (++h < h_kv) return;
        h = 0;
        do {
            if (++s >= B) return;  // behind the last unit
            n = prefix[s + 1] - prefix[s];
        } while (n == 0);
    }
};

// Row of S that entry s, with entry r of the slot map (without one: s), scores into on this step, -1 = none.
__device__ __forceinline__ int slot_of(const Q4Args &a, int s) { return a.score_rows ? __ldg(from_here(a.score_rows) + s) : s; }
__device__ __forceinline__ int q4_score_row(const Q4Args &a, int r, int L) {
    if (!a.want_score || L < 1 || (L - 1) % a.b < a.b - a.window) return -1;
    if (a.score_rows && r >= a.n_score_rows) {
        record_error(a.err, ZP_ERR_DEVICE, 0x15a);
        return -1;
    }
    return r < 0 ? -1 : r;
}

template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }

// After a wait that gave up at unit i of n: waits, for as long again at most, for the copies
// that are still under way (units i to i + stages - 1), so that none lands behind the kernel.
__device__ __noinline__ void drain(uint64_t *full, int stages, int i, int n) {
    const unsigned long long t0 = global_ns();
    for (int j = i; j < n && j < i + stages; ++j)
        while (!mbar_try_wait(&full[j % stages], (j / stages) & 1) && global_ns() - t0 < kWaitLimitNs) {
        }
}

// ---------------------------------------------------------------- records
// One pair's part in one range: per head float4 (reference, sum that divides the output, sum, 0),
// then the accumulators [G][D], all relative to 2^reference.  (Joined by the last CTA to arrive at a pair
// instead of by a second kernel, 1 x 32k took 28 us: 19 CTAs meet on its counter.)
__device__ __forceinline__ int rec_floats(const Q4Args &a, int d) { return a.G * (d + 4); }

// Normaliser of the score: p = 2^((logit - x) - y).  (Not in one number: far from zero the
// reference's step is larger than the logarithm.)  An empty sum gives no score.
__device__ __forceinline__ float2 score_norm(float m, float l) {
    return l == 0.f ? make_float2(INFINITY, 0.f) : make_float2(m, log2f(l));
}

// ---------------------------------------------------------------- tensor-core products
// Up to 8 q heads as the 8 columns of mma.sync m16n8k16: logits[t][h] with the key codes as the
// left operand, out^T[i][h] with the value codes.  (One kv head has 8 query rows at most: the 128
// rows of a tcgen05 tile would stand empty, and its operands would have to be written to shared
// memory at four times the size of the codes.)
//   logits:  sum_i q_i (lo + c_i step) = lo sum_i q_i + step sum_i q_i c_i per group.  The codes
//     go in as fp16 numbers without any arithmetic: the low nibble of a halfword, masked, is the
//     subnormal c 2^-24 and the next one c 2^-20 (whose queries are 2^-4 times as large), so that a
//     word of eight codes takes four masks and one shift.  The queries are scaled by a power of two
//     to fill fp16's range; those of 8 bits that lie within 2^-24 of the largest stay exact.  The
//     lo term is a product of its own, of the parameter words (step, lo) as they lie in the tile
//     with (0, sum q), the sum in three bf16 parts of 8 bits.  Nothing else is rounded to 16 bits:
//     the logits are those of 32-bit arithmetic.
//   output:  sum_t p_t lo_t + sum_t p_t step_t c_t.  The first is a product of p (two bf16 parts,
//     transposed by movmatrix) with the parameters as they are.  For the second p goes to fp16 and
//     its product with the step of a group to fp16 again, each off by 2^-11 of itself at most; the codes
//     are subnormals once more.  (Both in two fp16 parts: 64 sequences of 4k at most 56 us instead of
//     51, 512 365 instead of 324.  The output's own rounding is by up to 2^-8.)  For that a step's exponent
//     is moved by what suits an earlier unit.  A unit with steps far from that one's (p step needs
//     bf16's range) takes its products in bf16, p step in two parts that are off by 2^-15 at most, with
//     codes 0x4300 | c = 128 + c less 128, and the next units' exponents are moved by what suits it.  The
//     sum that divides is that of p in two bf16 parts (2^-17).
//   fp32 queries: three parts of 8 bits of the query for the logits; for the output p and p step in
//     three bf16 parts each, with codes c - 8 and the parameters' sum of lo + 8 step, and every
//     unit's products are summed from zero and added to the accumulators in 32 bits, since the
//     tensor core's own additions cut what they drop.  (64 sequences of 2k tokens at most: 57 us,
//     with 32-bit FMAs 98.)
// ldmatrix of a natural row of codes gives lane 4t + j the word j of a 16-byte chunk of
// token t, the layout of the left operand; its transposed form gives the codes of two
// adjacent tokens for 4 dimensions, the layout of the transposed values.
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same in fp16
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// products over 8 instead of 16
__device__ __forceinline__ void mma8_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(b0));
}
__device__ __forceinline__ void mma8_bf16_0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, {%7, %7, %7, %7};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(b0), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint32_t mul_bf2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t fma_bf2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ uint32_t f2_to_h2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// code E of two tokens as the bf16 numbers c - CENTRE (0 or 8): (128 + c) - (128 + CENTRE), all exact
template <int E, int CENTRE>
__device__ __forceinline__ uint32_t codes(uint32_t w) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w >> (4 * E)), "r"(0x000F000Fu), "r"(0x43004300u));  // (a & b) | c
    asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(r) : "r"(CENTRE ? 0xC308C308u : 0xC300C300u));
    return r;
}
// N words of shared memory, N of 1, 2, 4
template <int N>
__device__ __forceinline__ void lds(const uint32_t *p, uint32_t (&w)[N]) {
    if constexpr (N == 4) {
        const uint4 x = *reinterpret_cast<const uint4 *>(p);
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    } else if constexpr (N == 2) {
        const uint2 x = *reinterpret_cast<const uint2 *>(p);
        w[0] = x.x, w[1] = x.y;
    } else {
        w[0] = *p;
    }
}

// Probabilities are kept relative to 2^(m - kScale), and m follows the maximum when that passes
// it by kLazyMax: they stay below 2^15, so that fp16 holds them, with 11 bits down to 2^-14, that
// is 2^-25 of 2^m's, and nothing above 2^-36 of that goes to zero.  Far from zero, where a float's
// step is some units, m - kScale is rounded up and m + kLazyMax down: their distance, the exponent of
// the largest weight, is never above 15.  (m = base + kScale rounded down is m again, or a step above
// at a power of two, for which base is the same.)
constexpr float kLazyMax = 4.f, kScale = 11.f;
// Steps that a group's value products take in fp16: kWindow exponents, from kBelow under the largest step
// of some unit on, but none below 2^-34 (kLowest): the accumulators then hold no more than the sums
// they stand for (rescale).  The unit is a range's first, then every one with a live step outside.
constexpr int kBelow = 10, kWindow = 14, kLowest = 127 - 34;
constexpr uint32_t kNoWindow = 0xFFFFFFFFu;  // no unit yet
// byte g of `wins` for a largest step of exponent `top`
__device__ __forceinline__ uint32_t window_for(int top) { return min(max(top - kBelow, kLowest), 255 - kWindow) - 1; }

// x, y as the sum of N bf16 pairs
template <int N>
__device__ __forceinline__ void split_bf2(float x, float y, uint32_t (&part)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        part[i] = f2_to_bf2(x, y);
        const float2 f = bf2_to_f2(part[i]);
        x -= f.x;
        y -= f.y;
    }
}

template <typename T_, int D, int LG>
struct TcWarp {
    using T = T_;
    static constexpr bool kF32 = sizeof(T) == 4;
    static constexpr int kD = D, kWarps = kF32 ? 12 : 16;
    static constexpr int kTile = q4_tile_bytes(D, 1 << LG), kSharedBytes = kF32 ? 0 : 512;
    static constexpr int NG = D >> LG, kChunks = D / 32, kPerGroup = (1 << LG) / 32;  // chunks of a row, of a group
    static constexpr int kQ = kF32 ? 3 : 1;                                           // parts of a query
    uint32_t qb[kQ][kChunks][2][2];  // queries as the right operand, by part, chunk and half of its words
    uint32_t ob[3];  // (0, sum of the queries) of (head lane / 4, group lane % 4), in three parts, scaled as the products
    float unit_y[2];  // what a product is worth: log2(e) / sqrt(d) over the scale of heads 2 (lane % 4), + 1
    float acc[kChunks][2][4], off[4];
    float thr[2], base[2], l[2];  // of those two heads: m + kLazyMax (-inf: none yet), m - kScale, sum over this lane's tokens
    uint4 *params;     // bf16 queries: of a unit's values, by two tokens: steps in fp16 and lo in bf16, by group
    uint32_t wins;     // bf16 queries: by group a byte, lowest exponent, less 1, of the steps taken in fp16; or kNoWindow
    __device__ __forceinline__ uint32_t window(int g) const { return wins >> (8 * g) & 0xFFu; }

    struct Query {  // eight elements of each chunk
        uint4 w[kChunks][kF32 ? 2 : 1];
        __device__ __forceinline__ float get(int c, int i) const {
            if constexpr (kF32) return __uint_as_float((&w[c][i / 4].x)[i % 4]);
            const uint32_t x = (&w[c][0].x)[i / 2];
            return __uint_as_float(i % 2 ? x & 0xFFFF0000u : x << 16);
        }
    };
    static __device__ __forceinline__ Query fetch(const Q4Args &a, int s, int h, int lane) {
        const int n = lane >> 2, j = lane & 3;
        const T *q = from_here(static_cast<const T *>(a.q)) + ((size_t)s * a.h_q + (size_t)h * a.G + n) * D + j * 8;
        Query x;
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll
            for (int i = 0; i < (kF32 ? 2 : 1); ++i)
                x.w[c][i] = n < a.G ? __ldg(reinterpret_cast<const uint4 *>(q + c * 32) + i) : make_uint4(0, 0, 0, 0);
        return x;
    }
    __device__ __forceinline__ void begin(const Q4Args &a, const Query &x, int lane) {
        const int j = lane & 3;
        // the head's largest exponent (that of an infinity is one more than of any number)
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x.get(c, i)) & 0x7F800000u);
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        const int e = max((int)(top >> 23) - 127, -100);  // |q| < 2^(e + 1), scaled to below 2^15
        const float scale = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
        float sum[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) sum[g] = 0.f;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = x.get(c, i) * scale;
            sum[c / kPerGroup] += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
#pragma unroll
            for (int i = 1; i < 8; i += 2) v[i] *= 0.0625f;  // the elements of the high nibbles
#pragma unroll
            for (int k = 0; k < kQ; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float x0 = v[i], x1 = v[i + 4];
                    if constexpr (kF32) {  // 8 bits, whose products with the codes add up exactly
                        const float2 f = bf2_to_f2(f2_to_bf2(x0, x1));
                        x0 = f.x, x1 = f.y;
                        v[i] -= x0;
                        v[i + 4] -= x1;
                    }
                    qb[k][c][i / 2][i % 2] = f2_to_h2(x0, x1);
                }
        }
        float part = 0.f;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            sum[g] += __shfl_xor_sync(0xFFFFFFFFu, sum[g], 1);
            sum[g] += __shfl_xor_sync(0xFFFFFFFFu, sum[g], 2);
            if (j == g) part = sum[g] * 0x1p-24f;
        }
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const float hi = __bfloat162float(__float2bfloat16_rn(part));
            ob[i] = f2_to_bf2(0.f, hi);  // (lo is the high half of a parameter word, step the low one)
            part -= hi;
        }
        // 2^(24 - 14 + e) log2(e) / sqrt(d); an infinity (and the outputs NaN) for queries of 2^118 and more
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int eh = __shfl_sync(0xFFFFFFFFu, e, 8 * j + 4 * i);
            unit_y[i] = a.qscale * __uint_as_float((uint32_t)min(127 + eh + 10, 255) << 23);
        }
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[c][m][i] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) off[i] = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) thr[i] = -INFINITY, base[i] = 0.f, l[i] = 0.f;
        wins = kNoWindow;
    }

    // Two key tiles, then two value tiles; of tile i the tokens >= v0 (i = 0), v1 weigh nothing.
    __device__ __forceinline__ void unit(const Q4Args &a, unsigned char *tiles, int v0, int v1, float *logits, int lane) {
        const int n = lane >> 2, j = lane & 3;
        unsigned char *kt = tiles, *vt = tiles + 2 * kTile;
        const bool part = v0 + v1 < kUnit;
        if (part) {  // the parameters of the other tokens may be anything
            for (int i = lane; i < kUnit * NG; i += 32) {
                const int t = i / NG;
                if ((t & 15) < (t < kQ4Tile ? v0 : v1)) continue;
                const int at = t / kQ4Tile * kTile + q4_code_bytes(D) + (i % (kQ4Tile * NG)) * 4;
                *reinterpret_cast<uint32_t *>(kt + at) = *reinterpret_cast<uint32_t *>(vt + at) = 0;
            }
            fence_proxy_async_smem();  // (before the next copy into this stage)
            __syncwarp();
        }
        // rows and chunks of the four matrices of an ldmatrix: tokens 0-7 and 8-15 of one chunk, then of the next
        const int row = (lane & 7) + ((lane >> 3) & 1) * 8;
        const uint32_t at = row * (D / 2) + q4_chunk<D>(row, lane >> 4) * 16;
        // ---- logits of tokens n, n + 8 (of each tile) and heads 2j, 2j + 1
        float y[2][4];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const uint32_t *kp = reinterpret_cast<const uint32_t *>(kt + b * kTile + q4_code_bytes(D));
            const uint32_t p0 = NG == 4 || j < NG ? kp[n * NG + (NG == 4 ? j : j % NG)] : 0;
            const uint32_t p1 = NG == 4 || j < NG ? kp[(n + 8) * NG + (NG == 4 ? j : j % NG)] : 0;
            mma8_bf16_0(y[b], p0, p1, ob[2]);  // (small parts first)
            mma8_bf16(y[b], p0, p1, ob[1]);
            mma8_bf16(y[b], p0, p1, ob[0]);
            uint32_t w0[NG], w1[NG];
            lds<NG>(kp + n * NG, w0);
            lds<NG>(kp + (n + 8) * NG, w1);
            const uint32_t ka = smem_u32(kt + b * kTile) + at;
            float d[4];
#pragma unroll
            for (int c = 0; c < kChunks; c += 2) {
                uint32_t r[4];
                ldsm_x4(ka ^ (c << 4), r[0], r[1], r[2], r[3]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int g = (c + i) / kPerGroup;
                    uint32_t u[4], v[4];  // codes of words 0 and 1, 2 and 3 (nibbles) of tokens n, n + 8
                    nibbles(r[2 * i], u[0], u[2], v[0], v[2]);
                    nibbles(r[2 * i + 1], u[1], u[3], v[1], v[3]);
                    const auto &q = qb[0][c + i];
                    if constexpr (kF32) {
                        // the small parts together, then the two halves of the first by themselves:
                        // the tensor core's own additions cut what they drop
                        float d1[4], d2[4];
                        mma_f16_0(d, u[0], u[1], u[2], u[3], qb[kQ - 1][c + i][0][0], qb[kQ - 1][c + i][0][1]);
                        mma_f16(d, v[0], v[1], v[2], v[3], qb[kQ - 1][c + i][1][0], qb[kQ - 1][c + i][1][1]);
                        mma_f16(d, u[0], u[1], u[2], u[3], qb[kQ / 2][c + i][0][0], qb[kQ / 2][c + i][0][1]);
                        mma_f16(d, v[0], v[1], v[2], v[3], qb[kQ / 2][c + i][1][0], qb[kQ / 2][c + i][1][1]);
                        mma_f16_0(d1, u[0], u[1], u[2], u[3], q[0][0], q[0][1]);
                        mma_f16_0(d2, v[0], v[1], v[2], v[3], q[1][0], q[1][1]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) d[e] += d1[e] + d2[e];
                    } else {
                        if ((c + i) % kPerGroup == 0) mma_f16_0(d, u[0], u[1], u[2], u[3], q[0][0], q[0][1]);
                        else mma_f16(d, u[0], u[1], u[2], u[3], q[0][0], q[0][1]);
                        mma_f16(d, v[0], v[1], v[2], v[3], q[1][0], q[1][1]);
                    }
                    if (kF32 || (c + i + 1) % kPerGroup == 0) {
                        const float s0 = __uint_as_float(w0[g] << 16), s1 = __uint_as_float(w1[g] << 16);
                        y[b][0] = fmaf(s0, d[0], y[b][0]);
                        y[b][1] = fmaf(s0, d[1], y[b][1]);
                        y[b][2] = fmaf(s1, d[2], y[b][2]);
                        y[b][3] = fmaf(s1, d[3], y[b][3]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) y[b][i] *= unit_y[i & 1];
        }
        if (part) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int valid = b ? v1 : v0;
                if (n >= valid) y[b][0] = y[b][1] = -INFINITY;
                if (n + 8 >= valid) y[b][2] = y[b][3] = -INFINITY;
            }
        }
        if (logits) {
            const int h = 2 * j;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float *to = logits + (b * kQ4Tile + n) * a.G + h;
                if (a.G % 2 == 0) {
                    if (h < a.G) {
                        *reinterpret_cast<float2 *>(to) = make_float2(y[b][0], y[b][1]);
                        *reinterpret_cast<float2 *>(to + 8 * a.G) = make_float2(y[b][2], y[b][3]);
                    }
                    continue;
                }
                if (h < a.G) to[0] = y[b][0], to[8 * a.G] = y[b][2];
                if (h + 1 < a.G) to[1] = y[b][1], to[8 * a.G + 1] = y[b][3];
            }
        }
        // ---- softmax relative to a reference that is changed only when a logit passes it by far
        const float top0 = fmaxf(fmaxf(y[0][0], y[0][2]), fmaxf(y[1][0], y[1][2]));
        const float top1 = fmaxf(fmaxf(y[0][1], y[0][3]), fmaxf(y[1][1], y[1][3]));
        if (__any_sync(0xFFFFFFFFu, top0 > thr[0] || top1 > thr[1])) {
            float top[2] = {top0, top1};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], o));
                const float m = thr[i] == -INFINITY ? top[i] : fmaxf(__fadd_rd(base[i], kScale), top[i]);
                const float now = m == -INFINITY ? 0.f : __fsub_ru(m, kScale);
                const float alpha = thr[i] == -INFINITY ? 0.f : ex2_approx(base[i] - now);
                base[i] = now;
                thr[i] = __fadd_rd(m, kLazyMax);
                l[i] *= alpha;
                off[i] *= alpha;
                off[i + 2] *= alpha;
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
#pragma unroll
                    for (int e = 0; e < 2; ++e) acc[c][e][i] *= alpha, acc[c][e][i + 2] *= alpha;
            }
        }
        if constexpr (kF32) values_f32(vt, y, at, lane);
        else values_bf16(vt, y, v0, v1, at, lane);
    }

    // The nibbles of a word as fp16 pairs: c 2^-24 of nibbles 0, 4 and 2, 6 (a, c), c 2^-20 of 1, 5
    // and 3, 7 (b, d).
    static __device__ __forceinline__ void nibbles(uint32_t w, uint32_t &a, uint32_t &b, uint32_t &c, uint32_t &d) {
        a = w & 0x000F000Fu;
        b = w & 0x00F000F0u;
        c = w >> 8 & 0x000F000Fu;
        d = w >> 8 & 0x00F000F0u;
    }
    // the left operand of the sums with the parameters: rows g and 8 + g (lo, step) of group g, row 7 ones
    static __device__ __forceinline__ void parameter_rows(const uint32_t *vp, int n, int j, uint32_t (&w)[4]) {
        const bool in = n < NG;
        const uint32_t *q0 = vp + 2 * j * NG + (in ? n : 0);
        const uint32_t x0 = q0[0], x1 = q0[NG], x8 = q0[8 * NG], x9 = q0[9 * NG];
        const uint32_t rest = n == 7 ? 0x3F803F80u : 0;  // 1
        w[0] = in ? __byte_perm(x0, x1, 0x7632) : rest;
        w[1] = __byte_perm(x0, x1, 0x5410);
        w[2] = in ? __byte_perm(x8, x9, 0x7632) : rest;
        w[3] = __byte_perm(x8, x9, 0x5410);
    }
    // codes of tokens 2j, 2j + 1 (x0) and + 8 (x1), dimensions 4n + E and 4n + E + 1 of a chunk
    template <int E, int CENTRE>
    static __device__ __forceinline__ void code_rows(uint32_t x0, uint32_t x1, uint32_t (&w)[4]) {
        w[0] = codes<E, CENTRE>(x0), w[1] = codes<E + 1, CENTRE>(x0);
        w[2] = codes<E, CENTRE>(x1), w[3] = codes<E + 1, CENTRE>(x1);
    }

    // (The first unit's are chosen beside its other look at the steps: 256 short sequences 0.7 us less.)
    __device__ __forceinline__ void choose_windows(const unsigned char *vt, int v0, int v1, int lane) {
        uint32_t w[NG];
        lds<NG>(reinterpret_cast<const uint32_t *>(vt + (lane >> 4) * kTile + q4_code_bytes(D)) + (lane & 15) * NG, w);
        const bool live = (lane & 15) < (lane < kQ4Tile ? v0 : v1);
        wins = 0;
#pragma unroll
        for (int g = 0; g < NG; ++g)
            wins |= window_for((int)__reduce_max_sync(0xFFFFFFFFu, live ? w[g] & 0x7F80u : 0u) >> 7) << (8 * g);
    }

    // The accumulators of the value products in fp16 hold 2^(89 - e) times the sums of p step c (e:
    // the window's lowest exponent, kLowest = 93 or more), 16 times that for odd dimensions; to and
    // from sums of p step c.  Neither is larger than those sums, which are finite for values below 2^92:
    // windows of any lower exponent had let ordinary values pass the largest float after units of flat groups.
    // (In two factors: the power may be past the largest float.)
    __device__ __forceinline__ void rescale(bool plain) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int e = (int)window(c / kPerGroup) + 1 - 89, e0 = plain ? e : -e, half = e0 / 2;
            const float f = __uint_as_float((uint32_t)(127 + half) << 23), f2 = __uint_as_float((uint32_t)(127 + e0 - half) << 23);
            const float odd = plain ? 0.0625f * f2 : 16.f * f2;
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[c][m][i] = acc[c][m][i] * f * (i < 2 ? f2 : odd);
        }
    }

    __device__ __forceinline__ void values_bf16(const unsigned char *vt, const float (&y)[2][4], int v0, int v1, uint32_t at,
                                                int lane) {
        const int n = lane >> 2, j = lane & 3;
        // ---- lane t looks at token t: do the steps of all tokens lie in the window?  Two lanes then
        // lay out their two tokens' parameters, by group: steps in fp16 (bf16's bits with the exponent
        // moved and three zeros behind), lo as it is.  (Once per unit, not by each lane that needs them:
        // 512 sequences 340 -> 319 us.)
        bool wild;
        {
            uint32_t w[NG];
            lds<NG>(reinterpret_cast<const uint32_t *>(vt + (lane >> 4) * kTile + q4_code_bytes(D)) + (lane & 15) * NG, w);
            const bool live = (lane & 15) < (lane < kQ4Tile ? v0 : v1);
            if (wins == kNoWindow) {
                wins = 0;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const int top = (int)__reduce_max_sync(0xFFFFFFFFu, live ? w[g] & 0x7F80u : 0u) >> 7;
                    wins |= window_for(top) << (8 * g);
                }
            }
            bool out = false;
#pragma unroll
            for (int g = 0; g < NG; ++g) out |= (w[g] & 0xFFFFu) - ((window(g) + 1) << 7) >= (uint32_t)kWindow << 7;
            wild = __any_sync(0xFFFFFFFFu, live && out);
            uint32_t pair[4];
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                if (!live) w[g] = (window(g) + 1) << 7;  // (p = 0: any step whose fp16 form is a number)
                const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, w[g], 1);
                pair[g] = lane & 1 ? __byte_perm(w[g], other, 0x3276) : __byte_perm(w[g], other, 0x5410) * 8 - window(g) * (0x10001u << 10);
            }
            if constexpr (NG == 4) params[lane] = make_uint4(pair[0], pair[1], pair[2], pair[3]);
            else if constexpr (NG == 2) *reinterpret_cast<uint2 *>(params + lane) = make_uint2(pair[0], pair[1]);
            else *reinterpret_cast<uint32_t *>(params + lane) = pair[0];
            __syncwarp();
        }
        float p[2][4];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
            for (int i = 0; i < 4; ++i) p[b][i] = ex2_approx(y[b][i] - base[i & 1]);
            l[0] += p[b][0] + p[b][2];
            l[1] += p[b][1] + p[b][3];
            // the sums with lo, p in two bf16 parts: rows g of the left operand lo of group g, row 7 ones
            const uint32_t *q0 = reinterpret_cast<const uint32_t *>(params + b * 16 + 2 * j + 1) + (n < NG ? n : 0);
            const uint32_t rest = n == 7 ? 0x3F803F80u : 0;
            const uint32_t l0 = n < NG ? q0[0] : rest, l1 = n < NG ? q0[32] : rest;
            uint32_t u0[2], u1[2];
            split_bf2(p[b][0], p[b][1], u0);
            split_bf2(p[b][2], p[b][3], u1);
#pragma unroll
            for (int k = 1; k >= 0; --k) mma_bf16(off, l0, l0, l1, l1, transpose8(u0[k]), transpose8(u1[k]));
        }
        if (wild) {
            rescale(true);
            values_wide(vt, p, at, lane);
            choose_windows(vt, v0, v1, lane);
            rescale(false);
            return;
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            // right operand of the values' products: tokens 2j, 2j + 1 (and + 8) of head n
            const uint32_t b0 = transpose8(f2_to_h2(p[b][0], p[b][1])), b1 = transpose8(f2_to_h2(p[b][2], p[b][3]));
            uint32_t w0[NG], w1[NG];
            lds<NG>(reinterpret_cast<const uint32_t *>(params + b * 16 + 2 * j), w0);
            lds<NG>(reinterpret_cast<const uint32_t *>(params + b * 16 + 2 * j + 8), w1);
            const uint32_t va = smem_u32(vt + b * kTile) + at;
            uint32_t s0 = 0, s1 = 0;
#pragma unroll
            for (int c = 0; c < kChunks; c += 2) {
                uint32_t r[4];
                ldsm_x4_t(va ^ (c << 4), r[0], r[1], r[2], r[3]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int g = (c + i) / kPerGroup;
                    if ((c + i) % kPerGroup == 0) {
                        s0 = mul_h2(b0, w0[g]);
                        s1 = mul_h2(b1, w1[g]);
                    }
                    uint32_t x[4], z[4];
                    nibbles(r[2 * i], x[0], x[1], z[0], z[1]);
                    nibbles(r[2 * i + 1], x[2], x[3], z[2], z[3]);
                    mma_f16(acc[c + i][0], x[0], x[1], x[2], x[3], s0, s1);
                    mma_f16(acc[c + i][1], z[0], z[1], z[2], z[3], s0, s1);
                }
            }
        }
    }

    // The values' products where steps of any size meet: p step in two bf16 parts, the codes as bf16 numbers.
    __device__ __forceinline__ void values_wide(const unsigned char *vt, const float (&p)[2][4], uint32_t at, int lane) {
        const int j = lane & 3;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            uint32_t u0[2], u1[2];
            split_bf2(p[b][0], p[b][1], u0);
            split_bf2(p[b][2], p[b][3], u1);
            const uint32_t b0 = transpose8(u0[0]), b1 = transpose8(u1[0]), e0 = transpose8(u0[1]), e1 = transpose8(u1[1]);
            const uint32_t *vp = reinterpret_cast<const uint32_t *>(vt + b * kTile + q4_code_bytes(D)) + 2 * j * NG;
            const uint32_t va = smem_u32(vt + b * kTile) + at;
#pragma unroll
            for (int c = 0; c < kChunks; c += 2) {
                uint32_t r[4];
                ldsm_x4_t(va ^ (c << 4), r[0], r[1], r[2], r[3]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int g = (c + i) / kPerGroup;
                    const uint32_t w0 = __byte_perm(vp[g], vp[NG + g], 0x5410), w1 = __byte_perm(vp[8 * NG + g], vp[9 * NG + g], 0x5410);
                    uint32_t s0 = mul_bf2(b0, w0), s1 = mul_bf2(b1, w1);
#pragma unroll 1
                    for (int k = 0; k < 2; ++k) {
                        uint32_t w[4];
                        code_rows<0, 0>(r[2 * i], r[2 * i + 1], w);
                        mma_bf16(acc[c + i][0], w[0], w[1], w[2], w[3], s0, s1);
                        code_rows<2, 0>(r[2 * i], r[2 * i + 1], w);
                        mma_bf16(acc[c + i][1], w[0], w[1], w[2], w[3], s0, s1);
                        // what is left (b w - s is a number of bf16); one copy of the code, seldom run
                        s0 = fma_bf2(e0, w0, fma_bf2(b0, w0, s0 ^ 0x80008000u));
                        s1 = fma_bf2(e1, w1, fma_bf2(b1, w1, s1 ^ 0x80008000u));
                    }
                }
            }
        }
    }

    __device__ __forceinline__ void values_f32(const unsigned char *vt, const float (&y)[2][4], uint32_t at, int lane) {
        constexpr int kP = 3;  // parts of a probability
        const int n = lane >> 2, j = lane & 3;
        float p[2][4], d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
            for (int i = 0; i < 4; ++i) p[b][i] = ex2_approx(y[b][i] - base[i & 1]);
            l[0] += p[b][0] + p[b][2];
            l[1] += p[b][1] + p[b][3];
            uint32_t w[4], u0[kP], u1[kP];
            parameter_rows(reinterpret_cast<const uint32_t *>(vt + b * kTile + q4_code_bytes(D)), n, j, w);
            split_bf2(p[b][0], p[b][1], u0);
            split_bf2(p[b][2], p[b][3], u1);
#pragma unroll
            for (int k = kP - 1; k >= 0; --k) mma_bf16(d, w[0], w[1], w[2], w[3], transpose8(u0[k]), transpose8(u1[k]));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) off[i] += d[i];
        const uint32_t va = smem_u32(vt) + at;
        uint32_t r[2][4], s0[2][kP], s1[2][kP];
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            uint32_t w[2][2][4];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                if (c % 2 == 0) ldsm_x4_t((va + b * kTile) ^ (c << 4), r[b][0], r[b][1], r[b][2], r[b][3]);
                if (c % kPerGroup == 0) {
                    const uint32_t *vp = reinterpret_cast<const uint32_t *>(vt + b * kTile + q4_code_bytes(D)) + c / kPerGroup;
                    const float t0 = __uint_as_float(vp[n * NG] << 16), t1 = __uint_as_float(vp[(n + 8) * NG] << 16);
                    split_bf2(p[b][0] * t0, p[b][1] * t0, s0[b]);
                    split_bf2(p[b][2] * t1, p[b][3] * t1, s1[b]);
#pragma unroll
                    for (int k = 0; k < kP; ++k) s0[b][k] = transpose8(s0[b][k]), s1[b][k] = transpose8(s1[b][k]);
                }
                code_rows<0, 8>(r[b][2 * (c % 2)], r[b][2 * (c % 2) + 1], w[b][0]);
                code_rows<2, 8>(r[b][2 * (c % 2)], r[b][2 * (c % 2) + 1], w[b][1]);
            }
            float e[2][4] = {};
#pragma unroll
            for (int k = kP - 1; k >= 0; --k)  // small parts first
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int m = 0; m < 2; ++m) mma_bf16(e[m], w[b][m][0], w[b][m][1], w[b][m][2], w[b][m][3], s0[b][k], s1[b][k]);
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[c][m][i] += e[m][i];
        }
    }

    // heads 2j, 2j + 1: dimensions 32c + 4n .. + 3 in acc[c], the sums of the rounded p in off[2..3] and of p in l
    __device__ __forceinline__ void end(int lane) {
        const int j = lane & 3;
        if constexpr (!kF32)
            rescale(true);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], o);
            const float both = kF32 ? fmaf(8.f, off[i + 2], off[i]) : off[i];  // of group lane / 4
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                const float add = __shfl_sync(0xFFFFFFFFu, both, 4 * (c / kPerGroup) + j);
#pragma unroll
                for (int e = 0; e < 2; ++e) acc[c][e][i] += add, acc[c][e][i + 2] += add;
            }
            off[i + 2] = __shfl_sync(0xFFFFFFFFu, off[i], 28 + j);
        }
    }
    __device__ __forceinline__ float reference(int i) const { return thr[i] == -INFINITY ? -INFINITY : base[i]; }
    __device__ __forceinline__ void write_out(const Q4Args &a, int s, int h, int lane) const {
        const int n = lane >> 2, j = lane & 3;
        T *out = static_cast<T *>(a.out) + ((size_t)s * a.h_q + (size_t)h * a.G) * D;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int g = 2 * j + i;
            if (g >= a.G) break;
            const float r = off[i + 2] == 0.f ? 0.f : 1.f / off[i + 2];
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                const float4 x = make_float4(acc[c][0][i] * r, acc[c][0][i + 2] * r, acc[c][1][i] * r, acc[c][1][i + 2] * r);
                T *to = out + g * D + c * 32 + n * 4;
                if constexpr (kF32) *reinterpret_cast<float4 *>(to) = x;
                else *reinterpret_cast<uint2 *>(to) = make_uint2(f2_to_bf2(x.x, x.y), f2_to_bf2(x.z, x.w));
            }
            if (a.want_score && n == 0) a.stats[(size_t)s * a.h_q + h * a.G + g] = score_norm(reference(i), l[i]);
        }
    }
    __device__ __forceinline__ void write_record(const Q4Args &a, float *rec, int lane) const {
        const int n = lane >> 2, j = lane & 3;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int g = 2 * j + i;
            if (g >= a.G) break;
            if (n == 0) reinterpret_cast<float4 *>(rec)[g] = make_float4(reference(i), off[i + 2], l[i], 0.f);
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
                *reinterpret_cast<float4 *>(rec + 4 * a.G + g * D + c * 32 + n * 4) =
                    make_float4(acc[c][0][i], acc[c][0][i + 2], acc[c][1][i], acc[c][1][i + 2]);
        }
    }
};

// ---------------------------------------------------------------- the score
constexpr int kScoreUnroll = 4;

__device__ __forceinline__ float less(float logit, float2 c) { return (logit - c.x) - c.y; }

// Every 32nd token from t to t1 of a pair: S += share * 2^max_q ((logit - c.x) - c.y), or = where `fresh` and
// at P.  G4: vectors of four heads (0: any number of heads).  All loads of a round are under way at once.
template <int G4>
__device__ __forceinline__ void score_tokens(const Q4Args &a, const float *lg, const float2 (&c)[8], float *S, int t, int t1,
                                             int P, bool fresh, float share) {
    for (; t < t1; t += 32 * kScoreUnroll) {
        float top[kScoreUnroll], old[kScoreUnroll];
        if constexpr (G4 > 0) {
            float4 v[kScoreUnroll][G4];
#pragma unroll
            for (int k = 0; k < kScoreUnroll; ++k)
#pragma unroll
                for (int i = 0; i < G4; ++i) {
                    const int tok = min(t + 32 * k, t1 - 1);
                    v[k][i] = __ldcg(reinterpret_cast<const float4 *>(lg) + (size_t)tok * G4 + i);
                }
#pragma unroll
            for (int k = 0; k < kScoreUnroll; ++k) {
                const int tok = min(t + 32 * k, t1 - 1);
                old[k] = fresh || tok == P ? 0.f : S[tok];
            }
#pragma unroll
            for (int k = 0; k < kScoreUnroll; ++k) {
                top[k] = -INFINITY;
#pragma unroll
                for (int i = 0; i < G4; ++i)
                    top[k] = fmaxf(fmaxf(top[k], fmaxf(less(v[k][i].x, c[4 * i]), less(v[k][i].y, c[4 * i + 1]))),
                                   fmaxf(less(v[k][i].z, c[4 * i + 2]), less(v[k][i].w, c[4 * i + 3])));
            }
        } else {
#pragma unroll
            for (int k = 0; k < kScoreUnroll; ++k) {
                const int tok = min(t + 32 * k, t1 - 1);
                top[k] = -INFINITY;
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (q < a.G) top[k] = fmaxf(top[k], less(__ldcg(lg + (size_t)tok * a.G + q), c[q]));
                old[k] = fresh || tok == P ? 0.f : S[tok];
            }
        }
#pragma unroll
        for (int k = 0; k < kScoreUnroll; ++k)
            if (t + 32 * k < t1) S[t + 32 * k] = fmaf(ex2_approx(top[k]), share, old[k]);
    }
}

// The score of tokens t0 to t1 of the pair (a sequence of L tokens, kv head h), whose logits are lg, in row `row` of
// S; lane q's norm is head q's normaliser.
__device__ __forceinline__ void score_part(const Q4Args &a, int h, int L, int row, const float *lg, float2 norm, int t0,
                                           int t1, int lane) {
    float2 c[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) c[q] = make_float2(__shfl_sync(0xFFFFFFFFu, norm.x, q), __shfl_sync(0xFFFFFFFFu, norm.y, q));
    const int P = L - 1;
    const bool fresh = P % a.b == a.b - a.window;
    const float share = 1.f / (float)a.window;
    float *S = a.score + ((size_t)row * a.h_kv + h) * a.score_stride;
    lg = from_here(lg);
    if (a.G == 4) score_tokens<1>(a, lg, c, S, t0 + lane, t1, P, fresh, share);
    else if (a.G == 8) score_tokens<2>(a, lg, c, S, t0 + lane, t1, P, fresh, share);
    else score_tokens<0>(a, lg, c, S, t0 + lane, t1, P, fresh, share);
}

// ---------------------------------------------------------------- attention
// Shared memory: rings (a warp's tiles; at its end the record of a pair that goes on behind its
// range), what a warp lays out for itself, records of pairs that began before a warp's range
// (written while the ring is in use; in the workspace where there is no room), prefix.
// Sixteen warps of 128 registers in bf16 (12 bytes spilled at d = 128 and groups of 32), twelve of 168 in
// fp32 (92) (10, 13 and 14 were slower for either), each with a ring of its own: no barrier between them, and 2 to 4 units (5 KB each at
// d = 128 and groups of 32) in flight per warp are 160 KB and more per SM.
template <class W>
__host__ __device__ inline size_t attention_smem(int stages, int tile, int B, int G, bool heads_here) {
    return (size_t)W::kWarps * ((size_t)stages * 4 * tile + W::kSharedBytes + (heads_here ? (size_t)G * (W::kD + 4) * 4 : 0)) + ((size_t)B + 1) * 4;
}

template <class W, bool CLUSTER>
__global__ void __launch_bounds__(W::kWarps * 32, 1) q4_attention_kernel(const Q4Args a) {
    constexpr int D = W::kD, kWarps = W::kWarps;
    using T = typename W::T;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ uint64_t full_s[kWarps][kMaxStages];
    __shared__ int sums_s[kWarps];
    __shared__ int head_s[kWarps], tail_s[kWarps];  // pair of a warp's records, -1 = none; kDone in head: its last unit is in
    __shared__ int abort_s;
    constexpr int kDone = 1 << 30;
    constexpr int kFirst = 1 << 10, kLast = 1 << 11, kScored = 1 << 12;  // a unit's notes, above the tokens of its two tiles
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rec_n = rec_floats(a, D), stages = a.stages;
    const size_t ring_bytes = (size_t)stages * 4 * a.tile;
    unsigned char *ring = smem + warp * ring_bytes;
    unsigned char *own = smem + kWarps * ring_bytes + warp * W::kSharedBytes, *behind = smem + kWarps * (ring_bytes + W::kSharedBytes);
    float *heads = a.heads_here ? reinterpret_cast<float *>(behind)
                                : a.rec + (size_t)(2 * a.grid + (int)blockIdx.x * kWarps) * rec_n;
    int *prefix = reinterpret_cast<int *>(behind + (a.heads_here ? (size_t)kWarps * rec_n * 4 : 0));
    if (lane < stages) mbar_init(&full_s[warp][lane], 2);
    if (lane == 0) head_s[warp] = tail_s[warp] = -1;
    if (tid == 0) abort_s = 0;
    fence_barrier_init();
    pdl_wait();
    // the units that are cut: of all pairs, or (cluster) of the one that this CTA's cluster has
    int units, cta = blockIdx.x;
    if constexpr (CLUSTER) {
        const int pair = cta / a.cluster;
        cta -= pair * a.cluster;
        units = units_of(q4_len(a, pair / a.h_kv));
        __syncthreads();  // (the initialisation)
    } else {
        unit_prefix(a, prefix, sums_s);  // (has the barrier behind the initialisation)
        if (blockIdx.x == 0)
            for (int s = tid; s <= a.B; s += blockDim.x) a.prefix[s] = prefix[s];
        units = prefix[a.B] * a.h_kv;
    }
    if (units == 0) return;
    const Split split = make_split(a, units, CLUSTER ? a.cluster : a.grid);
    const bool mine = cta < split.ctas && warp < split.per_cta;
    const int g = cta * split.per_cta + warp;
    const int x0 = mine ? split.start(g) : 0;
    const int n = mine ? split.start(g + 1) - x0 : 0;
    if (n > 0) {
        const uint64_t pol = l2_evict_first_policy();
        // Units go in windows of 32: lane i finds out about unit i of the window that is
        // being issued, and keeps it until the products get there.
        int put_tile[2] = {-1, -1}, put_meta = 0, put_pair = 0, meta = 0, pair = 0;
        auto look = [&](int i0) {
            meta = put_meta;
            pair = put_pair;
            if (i0 + lane >= n) return;
            Cursor c;
            if constexpr (CLUSTER) c.at(a, x0 + i0 + lane);
            else c.seek(prefix, a.B, a.h_kv, x0 + i0 + lane);
            put_pair = c.s * a.h_kv + c.h;
            int blk[2], sub[2];  // (read beside the length: a row of the table has an entry for every token below its stride)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int col = div_by(2 * c.u + b, a.tpb, a.inv_tpb);
                sub[b] = 2 * c.u + b - col * a.tpb;
                blk[b] = col < a.table_stride ? __ldg(from_here(a.table) + (size_t)c.s * a.table_stride + col) : -1;
            }
            const int slot = a.want_score ? slot_of(a, c.s) : -1;
            const int L = q4_len(a, c.s);
            put_meta = (c.u == 0 ? kFirst : 0) | (c.u == c.n - 1 ? kLast : 0);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int t = 2 * c.u + b, valid = min(kQ4Tile, L - t * kQ4Tile);
                put_tile[b] = -1;
                if (valid <= 0) continue;
                if (blk[b] >= 0 && blk[b] < a.n_total) {
                    put_tile[b] = (blk[b] * a.h_kv + c.h) * a.tpb + sub[b];
                    put_meta |= valid << (5 * b);
                } else {
                    record_error(a.err, ZP_ERR_DEVICE, 0x159);  // (its tokens weigh nothing)
                }
            }

            if (a.want_score && q4_score_row(a, slot, L) >= 0) put_meta |= kScored;
        };
        int put_st = 0;
        auto issue = [&](int i) {  // lanes 0 and 1: one tile of keys and values each
            if (i && (i & 31) == 0) look(i);
            const int t0 = __shfl_sync(0xFFFFFFFFu, put_tile[0], i & 31), t1 = __shfl_sync(0xFFFFFFFFu, put_tile[1], i & 31);
            if (lane < 2) {
                const int from = lane ? t1 : t0;
                uint64_t *bar = &full_s[warp][put_st];
                if (from >= 0) {
                    unsigned char *to = ring + (put_st * 4 + lane) * a.tile;
                    const size_t at = (size_t)(unsigned)from * (unsigned)a.tile;
                    mbar_arrive_expect_tx(bar, 2 * a.tile);
                    bulk_g2s(to, a.k + at, a.tile, bar, pol);
                    bulk_g2s(to + 2 * a.tile, a.v + at, a.tile, bar, pol);
                } else {
                    mbar_arrive(bar);
                }
            }
            put_st = put_st + 1 == stages ? 0 : put_st + 1;
        };
        look(0);
        // the queries of the first pair, ahead of the tiles
        const int first = __shfl_sync(0xFFFFFFFFu, put_pair, 0);
        const typename W::Query query = W::fetch(a, first / a.h_kv, first % a.h_kv, lane);
        for (int i = 0; i < n && i < stages; ++i) issue(i);
        meta = put_meta;
        pair = put_pair;

        W w;
        w.params = reinterpret_cast<uint4 *>(own);
        w.begin(a, query, lane);
        int st = 0;
        unsigned phase = 0;
        bool began = false;  // the pair's first unit is in this range
        for (int i = 0; i < n; ++i) {
            // (units 32 and on were looked up stages before; `look` has then moved the window before on)
            if (i && (i & 31) == 0) meta = put_meta, pair = put_pair;
            const int now = __shfl_sync(0xFFFFFFFFu, meta, i & 31);
            if (now & kFirst) {
                began = true;
                if (i) {
                    const int id = __shfl_sync(0xFFFFFFFFu, pair, i & 31);
                    w.begin(a, W::fetch(a, id / a.h_kv, id % a.h_kv, lane), lane);
                }
            }
            if (!mbar_wait_bounded(&full_s[warp][st], phase, a.err, &abort_s, 0x15b)) {
                drain(full_s[warp], stages, i, n);
                break;
            }
            float *lg = nullptr;
            if (now & kScored)
                lg = a.logits + ((CLUSTER ? (size_t)((int)blockIdx.x / a.cluster) * a.pair_units : 0) + x0 + i) * (kUnit * a.G);
            w.unit(a, ring + st * 4 * a.tile, now & 31, now >> 5 & 31, lg, lane);
            __syncwarp();
            if (i + stages < n) issue(i + stages);
            if (++st == stages) st = 0, phase ^= 1;
            if ((now & kLast) || i == n - 1) {
                const bool last = now & kLast;
                const int id = __shfl_sync(0xFFFFFFFFu, pair, i & 31);
                w.end(lane);
                if (last && began) {
                    w.write_out(a, id / a.h_kv, id % a.h_kv, lane);
                } else {
                    // (a pair that goes on behind the range is its last: the ring is empty then)
                    w.write_record(a, began ? reinterpret_cast<float *>(ring) : heads + warp * rec_n, lane);
                    if (lane == 0) {
                        if (began) tail_s[warp] = id;
                        else head_s[warp] = id | (last ? kDone : 0);
                    }
                }
            }
        }
    }
    __syncthreads();
    if (!CLUSTER && abort_s) return;  // (the others of a cluster read this CTA's shared memory: it stays)
    // ---- the records of this CTA: a pair's chain begins in a warp's tail, or before the CTA in
    // the first warp's head, and goes on in the heads of the next warps.  A warp joins one head
    // of one chain at a time.
    const int my_head = lane < split.per_cta ? head_s[lane] : -1;
    const unsigned tails = __ballot_sync(0xFFFFFFFFu, lane < split.per_cta && tail_s[lane] >= 0);
    const int before = head_s[0] >= 0, chains = before + __popc(tails);
    // a cluster's CTA leaves its record in the last ring (empty by now; the one tail there is lies in the first)
    float *joined = reinterpret_cast<float *>(smem + (kWarps - 1) * ring_bytes);
    for (int task = warp; task < chains * a.G; task += kWarps) {
        const int chain = task / a.G, q = task - chain * a.G;
        const bool side = chain >= before;  // it begins in this CTA
        int w0 = 0;
        if (side) {
            unsigned rest = tails;
            for (int i = before; i < chain; ++i) rest &= rest - 1;
            w0 = __ffs(rest) - 1;
        }
        const int pair = (side ? tail_s[w0] : head_s[0]) & ~kDone;
        const unsigned same = __ballot_sync(0xFFFFFFFFu, lane > w0 && my_head >= 0 && (my_head & ~kDone) == pair);
        const int w1 = w0 + __ffs(~(same >> (w0 + 1))) - 1;  // the pair's last warp here
        const bool done = w1 > w0 || !side ? (head_s[w1] & kDone) != 0 : false;
        const float *rec0 = side ? reinterpret_cast<const float *>(smem + w0 * ring_bytes) : heads;
        auto rec = [&](int w) { return w == w0 ? rec0 : heads + w * rec_n; };
        const int s = pair / a.h_kv, h = pair % a.h_kv;
        float m = -INFINITY;
#pragma unroll 4
        for (int w = w0; w <= w1; ++w) m = fmaxf(m, rec(w)[4 * q]);
        const float base = m == -INFINITY ? 0.f : m;
        constexpr int kOwn = D / 32;
        float x[kOwn] = {}, lo = 0.f, l = 0.f;
#pragma unroll 4
        for (int w = w0; w <= w1; ++w) {
            const float4 r = *reinterpret_cast<const float4 *>(rec(w) + 4 * q);
            const float *v = rec(w) + 4 * a.G + q * D + lane * kOwn;
            const float f = ex2_approx(r.x - base);
            lo = fmaf(r.y, f, lo);
            l = fmaf(r.z, f, l);
#pragma unroll
            for (int e = 0; e < kOwn; ++e) x[e] = fmaf(v[e], f, x[e]);
        }
        if (side && done) {
            const float r = lo == 0.f ? 0.f : 1.f / lo;
            T *out = static_cast<T *>(a.out) + ((size_t)s * a.h_q + (size_t)h * a.G + q) * D + lane * kOwn;
#pragma unroll
            for (int e = 0; e < kOwn; ++e) out[e] = from_f<T>(x[e] * r);
            if (a.want_score && lane == 0) a.stats[(size_t)s * a.h_q + h * a.G + q] = score_norm(m, l);
        } else {
            float *to = CLUSTER ? joined : a.rec + (size_t)(2 * blockIdx.x + side) * rec_n;
#pragma unroll
            for (int e = 0; e < kOwn; ++e) to[4 * a.G + q * D + lane * kOwn + e] = x[e];
            if (lane == 0) reinterpret_cast<float4 *>(to)[q] = make_float4(m, lo, l, 0.f);
        }
    }
    if constexpr (CLUSTER) {
        const int pair = (int)blockIdx.x / a.cluster, rank = (int)blockIdx.x % a.cluster, s = pair / a.h_kv, h = pair % a.h_kv;
        __shared__ float2 norm_s[8];
        float2 norm = make_float2(INFINITY, 0.f);  // of head `lane`
        if (split.ctas > 1) {
            // ---- the records of the cluster's CTAs, a warp per head; for a score every CTA needs every head's sum
            const auto cluster = cooperative_groups::this_cluster();
            cluster.sync();
            for (int q = warp; q < a.G; q += kWarps) {
                constexpr int kOwn = D / 32;
                const bool mine = q % a.cluster == rank;
                if (!mine && !a.want_score) continue;
                float4 r = make_float4(-INFINITY, 0.f, 0.f, 0.f);  // lane c: CTA c's
                if (lane < split.ctas) r = reinterpret_cast<const float4 *>(cluster.map_shared_rank(joined, lane))[q];
                float m = r.x;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
                const float f = ex2_approx(r.x - (m == -INFINITY ? 0.f : m));
                if (a.want_score) {
                    float l = r.z * f;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
                    if (lane == 0) norm_s[q] = score_norm(m, l);
                }
                if (!mine) continue;
                float lo = 0.f, x[kOwn] = {};
#pragma unroll 4
                for (int c = 0; c < split.ctas; ++c) {
                    const float *v = cluster.map_shared_rank(joined, c) + 4 * a.G + q * D + lane * kOwn;
                    const float fc = __shfl_sync(0xFFFFFFFFu, f, c);
                    lo = fmaf(__shfl_sync(0xFFFFFFFFu, r.y, c), fc, lo);
#pragma unroll
                    for (int e = 0; e < kOwn; ++e) x[e] = fmaf(v[e], fc, x[e]);
                }
                const float by = lo == 0.f ? 0.f : 1.f / lo;
                T *out = static_cast<T *>(a.out) + ((size_t)s * a.h_q + (size_t)h * a.G + q) * D + lane * kOwn;
#pragma unroll
                for (int e = 0; e < kOwn; ++e) out[e] = from_f<T>(x[e] * by);
            }
            cluster.sync();  // (no CTA goes while its record is read)
            if (lane < a.G) norm = norm_s[lane];
        } else if (a.want_score) {
            __syncthreads();  // (this CTA has left the sums of all heads)
            if (lane < a.G) norm = __ldcg(from_here(a.stats) + (size_t)s * a.h_q + h * a.G + lane);
        }
        if (!a.want_score || n <= 0 || abort_s) return;
        const int slot = slot_of(a, s), L = q4_len(a, s), row = q4_score_row(a, slot, L);
        if (row < 0) return;
        // ---- the score of the warp's own units
        score_part(a, h, L, row, a.logits + (size_t)pair * a.pair_units * (kUnit * a.G), norm, x0 * kUnit, min((x0 + n) * kUnit, L),
                   lane);
    }
}

// ---------------------------------------------------------------- what is left
// CTA c joins the records of the pair that its counterpart of the attention kernel began and
// did not finish, and forms the score of that one's units.  Bound by latencies: about 3 us behind the
// attention kernel without a score, 20 for 256 sequences of 4k tokens, whose logits (60 MB) and
// scores it reads; four tokens per lane at a time, and its statistics, length and slot in one go.
constexpr int kFinishThreads = 512;

// Record of CTA c of a pair cut between CTAs, which CTA c0 begins.
__device__ __forceinline__ const float *cta_record(const Q4Args &a, int c0, int c, int rec_n) {
    return a.rec + (size_t)(2 * c + (c == c0 ? 1 : 0)) * rec_n;
}

template <typename T, int D>
__global__ void __launch_bounds__(kFinishThreads, 1) q4_finish_kernel(const Q4Args a) {
    extern __shared__ int prefix[];
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rec_n = rec_floats(a, D);
    for (int s = tid; s <= a.B; s += kFinishThreads) prefix[s] = a.prefix[s];
    __syncthreads();
    if (prefix[a.B] == 0) return;
    const Split split = make_split(a, prefix[a.B] * a.h_kv, a.grid);
    const int c0 = blockIdx.x;
    if (c0 >= split.ctas) return;
    const int b0 = split.cta_start(c0), b1 = split.cta_start(c0 + 1);
    {
        Cursor cut;
        cut.seek(prefix, a.B, a.h_kv, b1 - 1);
        const int first = b1 - 1 - cut.u, last = first + cut.n - 1;
        if (first >= b0 && last >= b1) {
            const int c1 = split.cta_of(last), n = c1 - c0 + 1;
            T *out = static_cast<T *>(a.out) + ((size_t)cut.s * a.h_q + (size_t)cut.h * a.G) * D;
            for (int i = tid; i < a.G * D; i += kFinishThreads) {
                const int q = i / D;  // the warp's: lane c has the statistics of record c (of 32 at a time)
                float m = -INFINITY, x = 0.f, lo = 0.f;
                for (int at = 0; at < n; at += 32) {
                    const int c = c0 + at + lane;
                    float2 hd = make_float2(-INFINITY, 0.f);
                    if (c <= c1) hd = *reinterpret_cast<const float2 *>(cta_record(a, c0, c, rec_n) + 4 * q);
                    float top = fmaxf(hd.x, m);
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                    const float base = top == -INFINITY ? 0.f : top, keep = ex2_approx(m - base), f = ex2_approx(hd.x - base);
                    m = top;
                    x *= keep;
                    lo *= keep;
                    const int most = min(32, n - at);
#pragma unroll 8
                    for (int k = 0; k < most; ++k) {
                        const float fk = __shfl_sync(0xFFFFFFFFu, f, k);
                        lo = fmaf(__shfl_sync(0xFFFFFFFFu, hd.y, k), fk, lo);
                        x = fmaf(cta_record(a, c0, c0 + at + k, rec_n)[4 * a.G + i], fk, x);
                    }
                }
                out[i] = from_f<T>(lo == 0.f ? 0.f : x / lo);
            }
        }
    }
    if (!a.want_score) return;
    // ---- the score: warps take equal parts of the CTA's units, a lane one token at a time
    constexpr int kWarps = kFinishThreads / 32;
    const int x0 = b0 + (int)((long long)(b1 - b0) * warp / kWarps), x1 = b0 + (int)((long long)(b1 - b0) * (warp + 1) / kWarps);
    if (x0 == x1) return;
    Cursor cur;
    cur.seek(prefix, a.B, a.h_kv, x0);
    for (int x = x0; x < x1;) {
        const int units = min(cur.n - cur.u, x1 - x);  // the rest of this pair
        // three loads at once; normalisers of the heads: lane q has head q's
        float2 norm = lane < a.G ? __ldcg(from_here(a.stats) + (size_t)cur.s * a.h_q + cur.h * a.G + lane) : make_float2(INFINITY, 0.f);
        const int slot = slot_of(a, cur.s), L = q4_len(a, cur.s), row = q4_score_row(a, slot, L);
        if (row >= 0) {
            const int first = x - cur.u, last = first + cur.n - 1;
            if (first < b0 || last >= b1) {  // a pair that several CTAs share
                const int k0 = split.cta_of(first), k1 = split.cta_of(last);
                if (lane < a.G) {
                    float m = -INFINITY, l = 0.f;
#pragma unroll 8
                    for (int c = k0; c <= k1; ++c) m = fmaxf(m, cta_record(a, k0, c, rec_n)[4 * lane]);
                    const float base = m == -INFINITY ? 0.f : m;
#pragma unroll 8
                    for (int c = k0; c <= k1; ++c) {
                        const float4 hd = *reinterpret_cast<const float4 *>(cta_record(a, k0, c, rec_n) + 4 * lane);
                        l = fmaf(hd.z, ex2_approx(hd.x - base), l);
                    }
                    norm = score_norm(m, l);
                }
            }
            const int t0 = cur.u * kUnit;
            score_part(a, cur.h, L, row, a.logits + (size_t)first * kUnit * a.G, norm, t0, min(t0 + units * kUnit, L), lane);
        }
        x += units;
        cur.u += units - 1;
        cur.next(prefix, a.B, a.h_kv);
    }
}

// ---------------------------------------------------------------- host
struct Q4Plan {
    int grid, warps, stages;
    bool heads_here;
    size_t smem;
    size_t off_prefix, off_stats, off_rec, off_logits, total;
};

// f(W) for the warp type of a cache
template <typename T, typename F>
auto with_group(const zp_cache_desc *D, int group, F f) {
    if (D->head_dim == 128 && group == 32) return f(TcWarp<T, 128, 5>());
    if (D->head_dim == 128 && group == 64) return f(TcWarp<T, 128, 6>());
    if (D->head_dim == 128) return f(TcWarp<T, 128, 7>());
    if (group == 32) return f(TcWarp<T, 64, 5>());
    return f(TcWarp<T, 64, 6>());
}
template <typename F>
auto with_warp(const zp_cache_desc *D, int group, F f) {
    return D->dtype == ZP_BF16 ? with_group<__nv_bfloat16>(D, group, f) : with_group<float>(D, group, f);
}

zp_status q4_plan(const zp_cache_desc *D, int group, int B, int table_stride, int scored, const DeviceInfo &dev, Q4Plan *p) {
    zp_status rc = check_q4(D, group, "q4_decode");
    if (rc != ZP_OK) return rc;
    const int G = D->h_q / D->h_kv;
    if (G > 8) return fail(ZP_ERR_SHAPE, "q4_decode: h_q/h_kv %d > 8", G);
    if (B > kQ4MaxB) return fail(ZP_ERR_SHAPE, "q4_decode: B %d > %d", B, kQ4MaxB);
    if ((long long)B * table_stride * D->block_size > INT32_MAX)
        return fail(ZP_ERR_SHAPE, "q4_decode: B=%d rows of %d blocks of %d tokens exceed 32 bits", B, table_stride,
                    D->block_size);
    if (((long long)table_stride * D->block_size / kUnit + 1) * B * D->h_kv > INT32_MAX / 2)
        return fail(ZP_ERR_SHAPE, "q4_decode: B=%d rows of %d blocks and %d heads exceed 32-bit units", B, table_stride, D->h_kv);
    if ((long long)D->n_total_blocks * D->h_kv * (D->block_size / kQ4Tile) > INT32_MAX)
        return fail(ZP_ERR_SHAPE, "q4_decode: %d blocks of %d tokens and %d heads exceed 32-bit tiles", D->n_total_blocks,
                    D->block_size, D->h_kv);
    const int d = D->head_dim, tile = q4_tile_bytes(d, group);
    with_warp(D, group, [&](auto w) {
        using W = decltype(w);
        const size_t room = (size_t)dev.smem_optin - 1024;  // (beside 1 KB static)
        p->warps = W::kWarps;
        p->grid = dev.sm_count;
        // two units in flight at least; the records' place before a third
        p->heads_here = attention_smem<W>(2, tile, B, G, true) <= room;
        p->stages = kMaxStages;
        while (p->stages > 2 && attention_smem<W>(p->stages, tile, B, G, p->heads_here) > room) --p->stages;
        p->smem = attention_smem<W>(p->stages, tile, B, G, p->heads_here);
        return 0;
    });
    size_t off = 0;
    p->off_prefix = off;
    off = align_up(off + ((size_t)B + 1) * 4, 256);
    p->off_stats = off;
    off = align_up(off + (size_t)B * D->h_q * 8, 256);
    p->off_rec = off;
    off = align_up(off + (size_t)(2 + p->warps) * p->grid * G * (d + 4) * 4, 256);
    p->off_logits = off;
    if (scored) off += (size_t)B * align_up((size_t)table_stride * D->block_size, kUnit) * D->h_q * 4;
    p->total = off;
    return ZP_OK;
}

// With few pairs of few tokens at most (by the table's width; the lengths are on the GPU) every
// pair gets a cluster of CTAs of its own, which join their records in each other's shared memory and
// form the scores of their own units: no look at the other lengths, no second kernel.  A cluster is as large as gives its warps a unit each, or as fits
// the GPU, and pairs that may have more than three units per warp take the even cut: a long one
// among short ones would hold the others up.  Measured, cluster and even cut, with 8 kv heads of 128 in bf16:
//     16 sequences of 100 tokens       6.7 and  9.2 us,  of 500 9.6 and 13.8
//      1 of 1k 10.3, 11.0;  4 of 2k 12.6, 13.5;  1 of 4k 12.6, 12.7;  4 of 4k 13.6, 16.0
//     scored: 16 of 100 8.0, 11.1;  4 of 2k 14.5, 16.4;  16 of 500 in fp32 13.3, 18.5
//     16 of 2k (four units per warp)  16.5 and 19.5, but one of 2k in one CTA 15.2, cut evenly 11.4.
constexpr int kMaxCluster = 16, kClusterUnits = 3;

// Clusters of `size` CTAs that the GPU runs at once, 0 where it cannot.
template <class W>
int clusters_at_once(int size, size_t smem, int device) {
    static std::mutex mutex;
    static std::map<std::pair<int, int>, int> known;
    const auto kernel = q4_attention_kernel<W, true>;
    std::lock_guard<std::mutex> lock(mutex);
    const auto at = known.find({device, size});
    if (at != known.end()) return at->second;
    int n = 0;
    if (set_max_dynamic_smem(reinterpret_cast<const void *>(kernel), smem, "q4_decode: shared-memory attribute") != ZP_OK) return 0;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(size);
        cfg.blockDim = dim3(W::kWarps * 32);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = size;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
    }
    if (e != cudaSuccess) {
        n = 0;
        cudaGetLastError();
    }
    known[{device, size}] = n;
    return n;
}

// CTAs that each pair gets, 0 where the units of all pairs are better cut evenly.
template <class W>
int pick_cluster(const Q4Args &a, const Q4Plan &p, int device) {
    const long long pairs = (long long)a.B * a.h_kv, units = a.pair_units;
    if (pairs > p.grid) return 0;
    int size = 1;
    while (size < kMaxCluster && units > (long long)size * W::kWarps && pairs * 2 * size <= p.grid &&
           pairs <= clusters_at_once<W>(2 * size, p.smem, device))
        size *= 2;
    const long long most = (long long)size * W::kWarps * kClusterUnits;
    return units <= most ? size : 0;
}

template <class W>
zp_status launch_q4(Q4Args a, const Q4Plan &p, int device, cudaStream_t st) {
    a.cluster = pick_cluster<W>(a, p, device);
    a.inv_ranges = 0xFFFFFFFFu / (unsigned)((a.cluster ? a.cluster : p.grid) * p.warps) + 1;
    const auto kernel = a.cluster ? q4_attention_kernel<W, true> : q4_attention_kernel<W, false>;
    zp_status rc = set_max_dynamic_smem(reinterpret_cast<const void *>(kernel), p.smem, "q4_decode: shared-memory attribute");
    if (rc != ZP_OK) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.cluster ? a.B * a.h_kv * a.cluster : p.grid);
    cfg.blockDim = dim3(p.warps * 32);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.cluster > 1 ? 2 : 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    if (e != cudaSuccess) return cuda_fail(e, "q4_decode: attention launch");
    if (a.cluster) return ok();
    const auto finish = q4_finish_kernel<typename W::T, W::kD>;
    e = launch_dependent(finish, dim3(p.grid), dim3(kFinishThreads), ((size_t)a.B + 1) * 4, st, a);
    if (e != cudaSuccess) return cuda_fail(e, "q4_decode: finish launch");
    return ok();
}

}  // namespace
}  // namespace zp

using namespace zp;

extern "C" size_t zp_q4_decode_workspace_size(const zp_cache_desc *D, int32_t group, int32_t B, int32_t table_stride,
                                              int32_t scored) {
    if (check_q4(D, group, "q4_decode") != ZP_OK) return 0;
    if (B < 0 || table_stride < 0) {
        fail(ZP_ERR_INVALID_ARG, "q4_decode: B=%d table_stride=%d", B, table_stride);
        return 0;
    }
    DeviceInfo dev;
    if (device_info(&dev) != ZP_OK) return 0;
    Q4Plan p;
    return q4_plan(D, group, B, table_stride, scored, dev, &p) == ZP_OK ? p.total : 0;
}

extern "C" zp_status zp_q4_decode_attn(const zp_cache_desc *D, int32_t group, const void *q, const void *k_cache,
                                       const void *v_cache, const int32_t *block_table, int32_t table_stride,
                                       const int32_t *seq_lens, int32_t B, void *out, float *score_accum,
                                       const int32_t *score_rows, int32_t n_score_rows, int32_t window,
                                       void *workspace, size_t workspace_bytes, void *stream) {
    zp_status rc = check_q4(D, group, "q4_decode");
    if (rc != ZP_OK) return rc;
    if (B < 0 || table_stride < 0) return fail(ZP_ERR_INVALID_ARG, "q4_decode: B=%d table_stride=%d", B, table_stride);
    if (B == 0) return ok();
    if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !out || !workspace)
        return fail(ZP_ERR_INVALID_ARG, "q4_decode: NULL buffer");
    if (table_stride < 1) return fail(ZP_ERR_INVALID_ARG, "q4_decode: table_stride < 1");
    if (score_accum && (window < 1 || window > D->block_size))
        return fail(ZP_ERR_INVALID_ARG, "q4_decode: window %d outside [1, b=%d]", window, D->block_size);
    if (score_accum && score_rows && n_score_rows < 1)
        return fail(ZP_ERR_INVALID_ARG, "q4_decode: a slot map needs n_score_rows >= 1");
    if (((uintptr_t)q | (uintptr_t)k_cache | (uintptr_t)v_cache | (uintptr_t)out | (uintptr_t)score_accum |
         (uintptr_t)workspace) % 16)
        return fail(ZP_ERR_INVALID_ARG, "q4_decode: buffers must be 16-byte aligned");
    const uintptr_t q0 = (uintptr_t)q, o0 = (uintptr_t)out, q_bytes = (uintptr_t)B * D->h_q * D->head_dim * elem_bytes(D->dtype);
    if (q0 < o0 + q_bytes && o0 < q0 + q_bytes)
        return fail(ZP_ERR_INVALID_ARG, "q4_decode: out overlaps q (queries are read after outputs are written)");
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != ZP_OK) return rc;
    Q4Plan p;
    rc = q4_plan(D, group, B, table_stride, score_accum != nullptr, dev, &p);
    if (rc != ZP_OK) return rc;
    if (workspace_bytes < p.total)
        return fail(ZP_ERR_CAPACITY, "q4_decode: workspace %zu < %zu bytes", workspace_bytes, p.total);
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    Q4Args a = {};
    a.q = q;
    a.k = static_cast<const unsigned char *>(k_cache);
    a.v = static_cast<const unsigned char *>(v_cache);
    a.out = out;
    a.table = block_table;
    a.table_stride = table_stride;
    a.seq_lens = seq_lens;
    a.B = B;
    a.h_q = D->h_q;
    a.h_kv = D->h_kv;
    a.G = D->h_q / D->h_kv;
    a.b = D->block_size;
    a.n_total = D->n_total_blocks;
    a.tile = q4_tile_bytes(D->head_dim, group);
    a.tpb = D->block_size / kQ4Tile;
    a.inv_tpb = a.tpb == 1 ? 0u : 0xFFFFFFFFu / (unsigned)a.tpb + 1;
    a.qscale = (float)(1.4426950408889634 / sqrt((double)D->head_dim));
    a.want_score = score_accum != nullptr;
    a.window = window;
    a.score = score_accum;
    a.score_stride = (long long)table_stride * D->block_size;
    a.score_rows = score_accum ? score_rows : nullptr;
    a.n_score_rows = n_score_rows;
    a.prefix = reinterpret_cast<int *>(ws + p.off_prefix);
    a.stats = reinterpret_cast<float2 *>(ws + p.off_stats);
    a.rec = reinterpret_cast<float *>(ws + p.off_rec);
    a.logits = reinterpret_cast<float *>(ws + p.off_logits);
    a.grid = p.grid;
    a.warps = p.warps;
    a.stages = p.stages;
    a.heads_here = p.heads_here;
    a.pair_units = (int)(((long long)table_stride * D->block_size + kUnit - 1) / kUnit);
    a.err = dev.error_word;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return with_warp(D, group, [&](auto w) { return launch_q4<decltype(w)>(a, p, dev.device, st); });
}
