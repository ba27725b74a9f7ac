// q4_decode.cu -- paged GQA decode attention over a 4-bit cache, with the window score.
//
// For every sequence s and query head h (Zipage paper §3, §6; the score is App. C.2's):
//     out[s][h] = sum_{t<L_s} softmax_t(q[s][h] . k_t / sqrt(d)) v_t,
// k_t and v_t the values that the cache's codes stand for (q4_format.cuh).
//
// Work unit = one tile of 16 tokens of one kv head.  The units of all (sequence, kv head)
// pairs are laid one after another and every warp takes an equal contiguous range, so
// ragged lengths cannot unbalance the grid.  A warp copies the tiles of its range to a ring of
// its own in shared memory (bulk copies, one mbarrier per stage) and runs an online softmax in
// base 2 over them.  A pair that lies in one warp's range is written out by it; of the others
// every warp leaves a record (maximum, sum, accumulator) that q4_merge_kernel joins.  On window
// steps the logits (log2 units) go to scratch; with the final statistics q4_score_kernel turns
// them into probabilities, takes the maximum over the q heads and adds 1/w of it.
#include <math.h>

#include "q4_format.cuh"

namespace zp {
namespace {

constexpr int kQ4MaxB = 4096;
constexpr int kMinUnits = 4;  // units per warp below which fewer warps take part

struct Q4Args {
    const void *q;
    const unsigned char *k, *v;
    void *out;
    const int32_t *table;
    int table_stride;
    const int32_t *seq_lens;
    int B, h_q, h_kv, G, b, n_total;
    int lg_group, tile;
    float qscale;  // log2(e) / sqrt(d)
    int want_score, window;
    float *score;
    long long score_stride;
    const int32_t *score_rows;
    int n_score_rows;
    int *prefix;    // [B+1] units before each sequence (of one kv head)
    float2 *stats;  // [B][h_q] final (max, sum), log2 units
    float *rec;     // [2 * warps][G * (D + 2)]: per head max and sum, then the accumulators
    float *logits;  // [units][16][G]
    int grid, warps;  // CTAs of the attention kernel, warps of one
    unsigned *err;
};

// ---------------------------------------------------------------- the split
struct Split {
    long long U, W;  // units, ranges
    int per_cta;     // ranges of a CTA: its first warps take one each
    __device__ __forceinline__ long long start(long long g) const { return g * U / W; }
    // the range that holds unit x: the largest g with start(g) <= x
    __device__ __forceinline__ long long owner(long long x) const { return ((x + 1) * W - 1) / U; }
};

__device__ __forceinline__ Split make_split(const Q4Args &a, int units) {
    Split p;
    p.U = (long long)units * a.h_kv;
    const long long want = (p.U + (long long)kMinUnits * a.grid - 1) / ((long long)kMinUnits * a.grid);
    p.per_cta = (int)(want < 1 ? 1 : want > a.warps ? a.warps : want);
    p.W = (long long)p.per_cta * a.grid;
    return p;
}

__device__ __forceinline__ int q4_len(const Q4Args &a, int s) {
    const int L = __ldg(a.seq_lens + s);
    const long long cap = (long long)a.table_stride * a.b;
    if (L < 0 || L > cap) {
        record_error(a.err, ZP_ERR_DEVICE, 0x158);
        return L < 0 ? 0 : (int)cap;
    }
    return L;
}

// prefix[s] = units of the sequences before s; blockDim.x threads, a multiple of 32.
__device__ void unit_prefix(const Q4Args &a, int *prefix, int *warp_sum) {
    const int per = (a.B + blockDim.x - 1) / blockDim.x;
    const int s0 = min((int)threadIdx.x * per, a.B), s1 = min(s0 + per, a.B);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int mine = 0;
    for (int s = s0; s < s1; ++s) {
        const int n = (q4_len(a, s) + kQ4Tile - 1) / kQ4Tile;
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
    __device__ __forceinline__ void seek(const int *prefix, int B, int h_kv, long long x) {
        int lo = 0, hi = B - 1;
        while (lo < hi) {  // the last s with prefix[s] * h_kv <= x (it has units)
            const int mid = (lo + hi + 1) >> 1;
            if ((long long)prefix[mid] * h_kv <= x) lo = mid;
            else hi = mid - 1;
        }
        s = lo;
        n = prefix[s + 1] - prefix[s];
        const int in = (int)(x - (long long)prefix[s] * h_kv);
        h = in / n;
        u = in - h * n;
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

// Row of S that entry s scores into on this step, -1 = none.
__device__ __forceinline__ int q4_score_row(const Q4Args &a, int s, int L) {
    if (!a.want_score || L < 1 || (L - 1) % a.b < a.b - a.window) return -1;
    if (!a.score_rows) return s;
    const int r = __ldg(a.score_rows + s);
    if (r >= a.n_score_rows) {
        record_error(a.err, ZP_ERR_DEVICE, 0x15a);
        return -1;
    }
    return r < 0 ? -1 : r;
}

template <typename T> __device__ __forceinline__ float to_f(T x);
template <> __device__ __forceinline__ float to_f(float x) { return x; }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
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

// ---------------------------------------------------------------- fp32 products
// One warp, GP >= G heads.  Logits: lane t and lane t + 16 take half of the dimensions of
// token t each; values: every lane takes D/32 dimensions of all tokens.
template <typename T, int D, int GP>
struct ScalarWarp {
    static constexpr int kDims = D / 32;
    static constexpr int kSharedFloats = GP * D + kQ4Tile * GP;
    float m[GP], l[GP], acc[GP][kDims];
    float *q_s, *p_s;

    __device__ __forceinline__ void begin(const Q4Args &a, int s, int h, int lane) {
        const T *q = static_cast<const T *>(a.q) + ((size_t)s * a.h_q + (size_t)h * a.G) * D;
        __syncwarp();
        for (int i = lane; i < GP * D; i += 32) q_s[i] = i < a.G * D ? to_f(q[i]) : 0.f;
        __syncwarp();
#pragma unroll
        for (int g = 0; g < GP; ++g) {
            m[g] = -INFINITY;
            l[g] = 0.f;
#pragma unroll
            for (int j = 0; j < kDims; ++j) acc[g][j] = 0.f;
        }
    }

    // one tile; tokens >= valid weigh nothing
    __device__ __forceinline__ void tile(const Q4Args &a, const unsigned char *kt, const unsigned char *vt, int valid,
                                         float *logits, int lane) {
        const int t = lane & 15, half = lane >> 4;
        const int words = D >> a.lg_group;
        float x[GP];
#pragma unroll
        for (int g = 0; g < GP; ++g) x[g] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            const int chunk = half * (D / 64) + c;
            const uint4 w = *reinterpret_cast<const uint4 *>(kt + t * (D / 2) + q4_chunk<D>(t, chunk) * 16);
            const uint32_t par = reinterpret_cast<const uint32_t *>(kt + q4_code_bytes(D))[t * words + (chunk * 32 >> a.lg_group)];
            const float step = __uint_as_float(par << 16), lo = __uint_as_float(par & 0xFFFF0000u);
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int j = 0; j < 8; j += 4) {
                    float k[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) k[e] = fmaf((float)(ws[i] >> (4 * (j + e)) & 15u), step, lo);
#pragma unroll
                    for (int g = 0; g < GP; ++g) {
                        const float4 q = *reinterpret_cast<const float4 *>(q_s + g * D + chunk * 32 + i * 8 + j);
                        x[g] = fmaf(k[0], q.x, fmaf(k[1], q.y, fmaf(k[2], q.z, fmaf(k[3], q.w, x[g]))));
                    }
                }
            }
        }
        float alpha[GP];
#pragma unroll
        for (int g = 0; g < GP; ++g) {
            x[g] = (x[g] + __shfl_xor_sync(0xFFFFFFFFu, x[g], 16)) * a.qscale;
            if (t >= valid) x[g] = -INFINITY;
            float top = x[g];
#pragma unroll
            for (int o = 8; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            const float was = m[g];
            m[g] = fmaxf(was, top);
            const float base = m[g] == -INFINITY ? 0.f : m[g];
            alpha[g] = ex2_approx(was - base);
            const float p = ex2_approx(x[g] - base);
            l[g] = l[g] * alpha[g] + p;  // of token t only: the lanes' sums are added at the end
            if (half == 0) {
                p_s[t * GP + g] = p;
                if (logits && g < a.G) logits[t * a.G + g] = x[g];
            }
#pragma unroll
            for (int j = 0; j < kDims; ++j) acc[g][j] *= alpha[g];
        }
        __syncwarp();
        const int e0 = lane * kDims;
        for (int tt = 0; tt < valid; ++tt) {
            const unsigned char *row = vt + tt * (D / 2) + q4_chunk<D>(tt, e0 / 32) * 16 + (e0 % 32) / 2;
            const uint32_t w = kDims == 4 ? *reinterpret_cast<const uint16_t *>(row) : *row;
            const uint32_t par = reinterpret_cast<const uint32_t *>(vt + q4_code_bytes(D))[tt * words + (e0 >> a.lg_group)];
            const float step = __uint_as_float(par << 16), lo = __uint_as_float(par & 0xFFFF0000u);
            float v[kDims];
#pragma unroll
            for (int j = 0; j < kDims; ++j) v[j] = fmaf((float)(w >> (4 * j) & 15u), step, lo);
#pragma unroll
            for (int g = 0; g < GP; ++g) {
                const float p = p_s[tt * GP + g];
#pragma unroll
                for (int j = 0; j < kDims; ++j) acc[g][j] = fmaf(p, v[j], acc[g][j]);
            }
        }
        __syncwarp();
    }

    // sums over the lanes (both halves hold the same tokens' sums)
    __device__ __forceinline__ void end() {
#pragma unroll
        for (int g = 0; g < GP; ++g)
#pragma unroll
            for (int o = 8; o; o >>= 1) l[g] += __shfl_xor_sync(0xFFFFFFFFu, l[g], o);
    }
    __device__ __forceinline__ void write_out(const Q4Args &a, int s, int h, int lane) const {
        T *out = static_cast<T *>(a.out) + ((size_t)s * a.h_q + (size_t)h * a.G) * D;
#pragma unroll
        for (int g = 0; g < GP; ++g) {
            if (g >= a.G) break;
            const float r = l[g] == 0.f ? 0.f : 1.f / l[g];
#pragma unroll
            for (int j = 0; j < kDims; ++j) out[g * D + lane * kDims + j] = from_f<T>(acc[g][j] * r);
            if (a.want_score && lane == 0) a.stats[(size_t)s * a.h_q + h * a.G + g] = make_float2(m[g], l[g]);
        }
    }
    __device__ __forceinline__ void write_record(const Q4Args &a, float *rec, int lane) const {
#pragma unroll
        for (int g = 0; g < GP; ++g) {
            if (g >= a.G) break;
            if (lane == 0) reinterpret_cast<float2 *>(rec)[g] = make_float2(m[g], l[g]);
#pragma unroll
            for (int j = 0; j < kDims; ++j) rec[2 * a.G + g * D + lane * kDims + j] = acc[g][j];
        }
    }
};

// ---------------------------------------------------------------- attention
constexpr int kScalarWarps = 8, kScalarStages = 4;

template <typename T, int D, int GP>
__global__ void __launch_bounds__(kScalarWarps * 32) q4_scalar_kernel(const Q4Args a) {
    using Warp = ScalarWarp<T, D, GP>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ uint64_t full_s[kScalarWarps][kScalarStages];
    __shared__ int bad_s[kScalarWarps][kScalarStages], sums_s[kScalarWarps];
    __shared__ int abort_s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    unsigned char *ring = smem + (size_t)warp * kScalarStages * 2 * a.tile;
    float *mine = reinterpret_cast<float *>(smem + (size_t)kScalarWarps * kScalarStages * 2 * a.tile) + warp * Warp::kSharedFloats;
    int *prefix = reinterpret_cast<int *>(reinterpret_cast<float *>(smem + (size_t)kScalarWarps * kScalarStages * 2 * a.tile) +
                                          kScalarWarps * Warp::kSharedFloats);
    if (lane < kScalarStages) mbar_init(&full_s[warp][lane], 1);
    if (tid == 0) abort_s = 0;
    fence_barrier_init();
    unit_prefix(a, prefix, sums_s);  // (has the barrier behind the initialisation)
    if (blockIdx.x == 0)
        for (int s = tid; s <= a.B; s += blockDim.x) a.prefix[s] = prefix[s];
    const Split split = make_split(a, prefix[a.B]);
    if (warp >= split.per_cta || split.U == 0) return;
    const long long g = (long long)blockIdx.x * split.per_cta + warp;
    const long long x0 = split.start(g);
    const int n = (int)(split.start(g + 1) - x0);
    if (n == 0) return;
    const uint64_t pol = l2_evict_first_policy();

    Cursor put, get;
    put.seek(prefix, a.B, a.h_kv, x0);
    get = put;
    int ids = 0, ids_of = -1, ids_at = 0;  // lane i: block of unit ids_at + i of sequence ids_of
    const int tpb = a.b / kQ4Tile;
    auto issue = [&](int i) {
        if (put.s != ids_of || put.u < ids_at || put.u >= ids_at + 32) {
            ids_of = put.s;
            ids_at = put.u;
            const int u = put.u + lane;
            ids = u < put.n ? __ldg(a.table + (size_t)put.s * a.table_stride + u / tpb) : -1;
        }
        const int blk = __shfl_sync(0xFFFFFFFFu, ids, put.u - ids_at);
        const int st = i % kScalarStages;
        if (lane == 0) {
            const bool ok = blk >= 0 && blk < a.n_total;
            bad_s[warp][st] = !ok;
            if (ok) {
                const size_t off = (((size_t)blk * a.h_kv + put.h) * tpb + put.u % tpb) * a.tile;
                mbar_arrive_expect_tx(&full_s[warp][st], 2 * a.tile);
                bulk_g2s(ring + (size_t)st * 2 * a.tile, a.k + off, a.tile, &full_s[warp][st], pol);
                bulk_g2s(ring + (size_t)st * 2 * a.tile + a.tile, a.v + off, a.tile, &full_s[warp][st], pol);
            } else {
                record_error(a.err, ZP_ERR_DEVICE, 0x159);
                mbar_arrive(&full_s[warp][st]);
            }
        }
        put.next(prefix, a.B, a.h_kv);
    };
    for (int i = 0; i < n && i < kScalarStages; ++i) issue(i);

    Warp w;
    w.q_s = mine;
    w.p_s = mine + GP * D;
    int L = 0;
    bool scored = false;
    for (int i = 0; i < n; ++i) {
        if (i == 0 || get.u == 0) {
            if (i == 0 || get.h == 0) {
                L = q4_len(a, get.s);
                scored = q4_score_row(a, get.s, L) >= 0;
            }
            w.begin(a, get.s, get.h, lane);
        }
        const int st = i % kScalarStages;
        if (!mbar_wait_bounded(&full_s[warp][st], (i / kScalarStages) & 1, a.err, &abort_s, 0x15b)) {
            drain(full_s[warp], kScalarStages, i, n);
            return;
        }
        const int valid = bad_s[warp][st] ? 0 : min(kQ4Tile, L - get.u * kQ4Tile);
        const unsigned char *kt = ring + (size_t)st * 2 * a.tile;
        w.tile(a, kt, kt + a.tile, valid, scored ? a.logits + (size_t)(x0 + i) * kQ4Tile * a.G : nullptr, lane);
        __syncwarp();
        if (i + kScalarStages < n) issue(i + kScalarStages);
        const bool last = get.u == get.n - 1;
        if (last || i == n - 1) {
            w.end();
            const bool from_start = i >= get.u;  // the pair's first unit is in this range
            if (last && from_start) w.write_out(a, get.s, get.h, lane);
            else w.write_record(a, a.rec + (size_t)(2 * g + (from_start ? 1 : 0)) * a.G * (D + 2), lane);
        }
        get.next(prefix, a.B, a.h_kv);
    }
}

// ---------------------------------------------------------------- joining the records
// One CTA per pair that several ranges share: warp w takes every eighth record, then the
// warps are joined.
constexpr int kMergeWarps = 8;

template <typename T, int D>
__global__ void __launch_bounds__(kMergeWarps * 32) q4_merge_kernel(const Q4Args a) {
    extern __shared__ float sm[];  // [warps][G][D], [warps][G] (max, sum)
    pdl_wait();
    const int s = blockIdx.x / a.h_kv, h = blockIdx.x % a.h_kv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = a.prefix[s + 1] - a.prefix[s];
    if (n == 0) return;
    const Split split = make_split(a, a.prefix[a.B]);
    const long long p0 = (long long)a.prefix[s] * a.h_kv + (long long)h * n;
    const long long g0 = split.owner(p0), g1 = split.owner(p0 + n - 1);
    if (g0 == g1) return;
    const int stride = a.G * (D + 2);
    constexpr int kDims = D / 32;
    float *ml = sm + kMergeWarps * a.G * D;
    for (int g = 0; g < a.G; ++g) {
        float m = -INFINITY, l = 0.f, acc[kDims] = {};
        for (long long r = g0 + warp; r <= g1; r += kMergeWarps) {
            if (split.start(r) == split.start(r + 1)) continue;  // an empty range
            const float *rec = a.rec + (size_t)(2 * r + (split.start(r) <= p0 ? 1 : 0)) * stride;
            const float2 x = reinterpret_cast<const float2 *>(rec)[g];
            const float top = fmaxf(m, x.x), base = top == -INFINITY ? 0.f : top;
            const float was = ex2_approx(m - base), now = ex2_approx(x.x - base);
            m = top;
            l = l * was + x.y * now;
#pragma unroll
            for (int j = 0; j < kDims; ++j) acc[j] = acc[j] * was + rec[2 * a.G + g * D + lane * kDims + j] * now;
        }
#pragma unroll
        for (int j = 0; j < kDims; ++j) sm[(warp * a.G + g) * D + lane * kDims + j] = acc[j];
        if (lane == 0) {
            ml[(warp * a.G + g) * 2] = m;
            ml[(warp * a.G + g) * 2 + 1] = l;
        }
    }
    __syncthreads();
    T *out = static_cast<T *>(a.out) + ((size_t)s * a.h_q + (size_t)h * a.G) * D;
    for (int i = threadIdx.x; i < a.G * D; i += blockDim.x) {
        const int g = i / D;
        float m = -INFINITY, l = 0.f, acc = 0.f;
        for (int w = 0; w < kMergeWarps; ++w) m = fmaxf(m, ml[(w * a.G + g) * 2]);
        const float base = m == -INFINITY ? 0.f : m;
        for (int w = 0; w < kMergeWarps; ++w) {
            const float now = ex2_approx(ml[(w * a.G + g) * 2] - base);
            l += ml[(w * a.G + g) * 2 + 1] * now;
            acc += sm[w * a.G * D + i] * now;
        }
        out[i] = from_f<T>(l == 0.f ? 0.f : acc / l);
        if (a.want_score && i % D == 0) a.stats[(size_t)s * a.h_q + h * a.G + g] = make_float2(m, l);
    }
}

// ---------------------------------------------------------------- window score
// The units are split as for the attention; a half-warp takes one at a time, a lane a token.
constexpr int kScoreWarps = 8;

__global__ void __launch_bounds__(kScoreWarps * 32) q4_score_kernel(const Q4Args a) {
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = lane & 15, half = lane >> 4;
    const long long U = (long long)a.prefix[a.B] * a.h_kv, W = (long long)gridDim.x * kScoreWarps;
    const long long g = (long long)blockIdx.x * kScoreWarps + warp;
    const long long x0 = g * U / W, x1 = (g + 1) * U / W;
    if (x0 >= x1) return;
    Cursor c;
    c.seek(a.prefix, a.B, a.h_kv, x0);
    for (long long x = x0; x < x1;) {
        // the rest of this pair
        const int units = (int)min((long long)(c.n - c.u), x1 - x);
        const int L = q4_len(a, c.s), row = q4_score_row(a, c.s, L);
        if (row >= 0) {
            const int P = L - 1;
            const bool first = P % a.b == a.b - a.window;
            const float share = 1.f / (float)a.window;
            float *S = a.score + ((size_t)row * a.h_kv + c.h) * a.score_stride;
            const float2 *st = a.stats + (size_t)c.s * a.h_q + c.h * a.G;
            for (int i = half; i < units; i += 2) {
                const int tok = (c.u + i) * kQ4Tile + t;
                if (tok > P) continue;
                const float *lg = a.logits + ((size_t)(x + i) * kQ4Tile + t) * a.G;
                float top = 0.f;
                for (int q = 0; q < a.G; ++q) {
                    const float2 ml = st[q];
                    const float p = ml.y > 0.f ? ex2_approx(lg[q] - ml.x) / ml.y : 0.f;
                    top = fmaxf(top, p);
                }
                top *= share;
                S[tok] = first || tok == P ? top : S[tok] + top;
            }
        }
        x += units;
        c.u += units - 1;
        c.next(a.prefix, a.B, a.h_kv);
    }
}

// ---------------------------------------------------------------- host
struct Q4Plan {
    int grid, warps;
    size_t smem;
    size_t off_prefix, off_stats, off_rec, off_logits, total;
};

int padded_group(int G) { return G <= 1 ? 1 : G <= 2 ? 2 : G <= 4 ? 4 : 8; }

zp_status q4_plan(const zp_cache_desc *D, int group, int B, int table_stride, int scored, const DeviceInfo &dev, Q4Plan *p) {
    zp_status rc = check_q4(D, group, "q4_decode");
    if (rc != ZP_OK) return rc;
    const int G = D->h_q / D->h_kv;
    if (G > 8) return fail(ZP_ERR_SHAPE, "q4_decode: h_q/h_kv %d > 8", G);
    if (B > kQ4MaxB) return fail(ZP_ERR_SHAPE, "q4_decode: B %d > %d", B, kQ4MaxB);
    if ((long long)B * table_stride * D->block_size > INT32_MAX)
        return fail(ZP_ERR_SHAPE, "q4_decode: B=%d rows of %d blocks of %d tokens exceed 32 bits", B, table_stride,
                    D->block_size);
    const int d = D->head_dim, GP = padded_group(G), tile = q4_tile_bytes(d, group);
    p->warps = kScalarWarps;
    p->smem = (size_t)kScalarWarps * kScalarStages * 2 * tile + (size_t)kScalarWarps * (GP * d + kQ4Tile * GP) * 4 +
              ((size_t)B + 1) * 4;
    const int per_sm = (int)(dev.smem_optin / p->smem);
    p->grid = dev.sm_count * (per_sm < 1 ? 1 : per_sm > 2 ? 2 : per_sm);
    size_t off = 0;
    p->off_prefix = off;
    off = align_up(off + ((size_t)B + 1) * 4, 256);
    p->off_stats = off;
    off = align_up(off + (size_t)B * D->h_q * 8, 256);
    p->off_rec = off;
    off = align_up(off + (size_t)2 * p->grid * p->warps * G * (d + 2) * 4, 256);
    p->off_logits = off;
    if (scored) off = align_up(off + (size_t)B * table_stride * D->block_size * D->h_q * 4, 256);
    p->total = off;
    return ZP_OK;
}

template <typename T, int D, int GP>
zp_status launch_attention(const Q4Args &a, const Q4Plan &p, cudaStream_t st) {
    const auto kernel = q4_scalar_kernel<T, D, GP>;
    const zp_status rc = set_max_dynamic_smem(reinterpret_cast<const void *>(kernel), p.smem, "q4_decode: shared-memory attribute");
    if (rc != ZP_OK) return rc;
    kernel<<<p.grid, p.warps * 32, p.smem, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? ZP_OK : cuda_fail(e, "q4_decode: attention launch");
}

template <typename T, int D>
zp_status launch_q4(const Q4Args &a, const Q4Plan &p, cudaStream_t st) {
    zp_status rc;
    switch (padded_group(a.G)) {
        case 1: rc = launch_attention<T, D, 1>(a, p, st); break;
        case 2: rc = launch_attention<T, D, 2>(a, p, st); break;
        case 4: rc = launch_attention<T, D, 4>(a, p, st); break;
        default: rc = launch_attention<T, D, 8>(a, p, st); break;
    }
    if (rc != ZP_OK) return rc;
    const size_t smem = (size_t)kMergeWarps * a.G * (D + 2) * 4;
    const auto merge = q4_merge_kernel<T, D>;
    rc = set_max_dynamic_smem(reinterpret_cast<const void *>(merge), smem, "q4_decode: shared-memory attribute");
    if (rc != ZP_OK) return rc;
    cudaError_t e = launch_dependent(merge, dim3(a.B * a.h_kv), dim3(kMergeWarps * 32), smem, st, a);
    if (e != cudaSuccess) return cuda_fail(e, "q4_decode: merge launch");
    if (!a.want_score) return ok();
    e = launch_dependent(q4_score_kernel, dim3(4 * p.grid), dim3(kScoreWarps * 32), 0, st, a);
    if (e != cudaSuccess) return cuda_fail(e, "q4_decode: score launch");
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
    a.lg_group = group == 32 ? 5 : group == 64 ? 6 : 7;
    a.tile = q4_tile_bytes(D->head_dim, group);
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
    a.err = dev.error_word;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool wide = D->head_dim == 128;
    if (D->dtype == ZP_BF16) return wide ? launch_q4<__nv_bfloat16, 128>(a, p, st) : launch_q4<__nv_bfloat16, 64>(a, p, st);
    return wide ? launch_q4<float, 128>(a, p, st) : launch_q4<float, 64>(a, p, st);
}
