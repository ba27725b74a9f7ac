// prefix_common.cuh -- the work split of the prefix kernels (prefix_attn.cu,
// prefix_tc.cu): the groups of a plan, the tiles of their items and the places
// of their partial records.
#pragma once

#include "zp_common.cuh"

namespace zp {

constexpr int kPfxMaxB = 4096;

struct PfxArgs {
    const void *q, *k, *v;
    const int32_t *table;
    int stride;
    const int32_t *seq_lens;
    int B, h_q, h_kv, n_total;
    int b, b_log;        // tokens per block, a power of two
    int G, G_log;        // q heads per kv head, a power of two
    // the plan
    const int32_t *prefix, *n_groups, *group_start, *members, *group_blocks;
    int rt_log, kt_log;  // rows per item, tokens per tile (powers of two)
    int parts;           // sets of CTAs (split of the tiles); a set has a CTA per kv head
    float qscale;        // log2(e) / sqrt(d)
    int *wpre;           // [B+1] places before each group
    int *place;          // [B] place of every batch entry in the member list, -1 = in no group
    float *rec_acc;      // [extra0 + parts*rt][d] pieces: main records, then extra records
    float2 *rec_ml;      // same rows
    long long extra0;    // first extra record: B*h_q, twice that on the tensor cores (second streams);
                         // then rt rows per CTA (set * h_kv + head)
    int tc;              // tensor-core kernels: 256 rows x 128 tokens, two streams
    float *whole_acc;    // [B][h_q][d] the decode's records of sequences that one CTA saw whole
    float2 *whole_ml;    // [B][h_q]
    // score
    float *score;
    long long score_stride;
    const int32_t *score_rows;
    int n_score_rows, window;
    const float *stats;   // [B][h_q] final max + log2(sum)
    const float *logits;  // the decode's: [units][tokens of a unit][h_q], log2 units
    const int4 *units;    // [units] (sequence, first token, length behind the prefix, window flags)
    const int *n_units;   // [1]
    int unit_log;         // tokens of a unit, a power of two
    unsigned *err;
};

// Group g of the plan, with every index the plan gives bounded.
struct PfxGroup {
    int m0, n;    // first member, members
    int tokens;   // prefix tokens
    int rts, kts; // row tiles, token tiles
    int lead;     // places that an item's start takes in the split, beside its tiles'
};

// An item's start (its queries fetched with nothing to compute meanwhile, and the
// records of the item before written) costs a CTA as much as about five tiles on the
// tensor cores, so in the split of the work it has places of its own ahead of the
// tiles, at most one per eight tiles: a CTA that begins a second item gets fewer
// tiles.  (256 sequences behind two prefixes of 4k, four items of 32 tiles on 19 CTAs:
// the slowest CTA 22 us, 29 us without; scored in all 145, 151 us without.)  In fp32 a
// tile costs more than a start.
constexpr int kPfxLead = 4;

__device__ __forceinline__ int pfx_groups(const PfxArgs &a) { return min(max(__ldg(a.n_groups), 0), a.B); }

__device__ __forceinline__ PfxGroup pfx_group(const PfxArgs &a, int g) {
    PfxGroup r;
    r.m0 = min(max(__ldg(a.group_start + g), 0), a.B);
    r.n = min(max(__ldg(a.group_start + g + 1), r.m0), a.B) - r.m0;
    r.tokens = min(max(__ldg(a.group_blocks + g), 0), a.stride) << a.b_log;
    r.rts = ((r.n << a.G_log) + (1 << a.rt_log) - 1) >> a.rt_log;
    r.kts = (r.tokens + (1 << a.kt_log) - 1) >> a.kt_log;
    r.lead = a.tc ? min(kPfxLead, r.kts >> 3) : 0;
    return r;
}

// Places of a group in the split.
__device__ __forceinline__ int pfx_places(const PfxGroup &g) { return g.rts * (g.lead + g.kts); }

// Group of place i of the member list: the last that starts at or before it
// (ng > 0; the place may lie behind its end).
__device__ __forceinline__ int pfx_group_of(const PfxArgs &a, int ng, int i) {
    int lo = 0, hi = ng - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(a.group_start + mid) <= i) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Batch entry of member i; an entry outside the batch is recorded, -1.
__device__ __forceinline__ int pfx_member(const PfxArgs &a, int i) {
    const int s = __ldg(a.members + i);
    if (s < 0 || s >= a.B) {
        record_error(a.err, ZP_ERR_DEVICE, 0x142);
        return -1;
    }
    return s;
}

__device__ __forceinline__ int pfx_start(int c, int W, int parts) { return (int)((long long)c * W / parts); }

// last g in [0, n) with pre[g] <= x
__device__ __forceinline__ int pfx_find(const int *pre, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pre[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Set whose range holds tile w: the largest c with floor(c W / parts) <= w.
__device__ __forceinline__ int pfx_owner(int w, int W, int parts) {
    return (int)(((long long)(w + 1) * parts - 1) / W);
}

// Places before each group (whole CTA; pre: n_groups + 1 ints of shared memory);
// returns the total.
inline __device__ int pfx_scan(const PfxArgs &a, int ng, int *pre) {
    for (int i = threadIdx.x; i < ng; i += blockDim.x) pre[i] = pfx_places(pfx_group(a, i));
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int carry = 0;
        for (int base = 0; base < ng; base += 32) {
            const int x = base + lane < ng ? pre[base + lane] : 0;
            int v = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xFFFFFFFFu, v, o);
                if (lane >= o) v += y;
            }
            if (base + lane < ng) pre[base + lane] = carry + v - x;
            carry += __shfl_sync(0xFFFFFFFFu, v, 31);
        }
        if (lane == 0) pre[ng] = carry;
    }
    __syncthreads();
    return pre[ng];
}

// What a CTA does from place w of its range, which ends at w1: tiles [t_b, t_e) of row
// tile `item` of group g (none where its places end ahead of the first), up to place
// w_e.
struct PfxSeg {
    PfxGroup g;
    int item, t_b, t_e, w_e;
};

__device__ __forceinline__ PfxSeg pfx_segment(const PfxArgs &a, const int *pre, int ng, int w, int w1) {
    PfxSeg s;
    const int gi = pfx_find(pre, ng, w);
    s.g = pfx_group(a, gi);
    const int x = w - pre[gi], len = s.g.lead + s.g.kts;
    s.item = (int)((unsigned)x / (unsigned)len);
    const int at = x - s.item * len, end = min(len, at + (w1 - w));
    s.t_b = max(at - s.g.lead, 0);
    s.t_e = max(end - s.g.lead, 0);
    s.w_e = w + (end - at);
    return s;
}

// Row of the main records: rows of a group are (kv head, member, q head of the
// group), after the rows of the members before it.
__device__ __forceinline__ long long pfx_main_row(const PfxArgs &a, const PfxGroup &g, int head, int r) {
    return (long long)g.m0 * a.h_q + (long long)head * (g.n << a.G_log) + r;
}

// Physical row (block * b + slot) of token t of the group's prefix, by its first
// member's table row; -1 for a bad block id (recorded).
__device__ __forceinline__ long long pfx_slot(const PfxArgs &a, const int32_t *row, int t) {
    const int blk = __ldg(row + (t >> a.b_log));
    if (blk < 0 || blk >= a.n_total) {
        record_error(a.err, ZP_ERR_DEVICE, 0x143);
        return -1;
    }
    return ((long long)blk << a.b_log) + (t & (a.b - 1));
}

// The table row every member's prefix agrees with: that of the first member inside
// the batch (row 0 if there is none: nobody reads the group's records then).
__device__ __forceinline__ const int32_t *pfx_row(const PfxArgs &a, const PfxGroup &g) {
    int s = -1;
    for (int i = g.m0; s < 0 && i < g.m0 + g.n; ++i) s = pfx_member(a, i);
    return a.table + (size_t)max(s, 0) * a.stride;
}

// Row of the score that batch entry s adds to in this step, -1: none (no prefix,
// not on a window step, no score row).  first: the window's first row, written.
__device__ __forceinline__ int pfx_score_row(const PfxArgs &a, int s, bool *first) {
    const int L = min(__ldg(a.seq_lens + s), a.stride * a.b);
    const int p = __ldg(a.prefix + s);
    *first = false;
    if (p <= 0 || p >= L || (p & (a.b - 1))) return -1;
    const int ph = (L - 1) & (a.b - 1);
    if (ph < a.b - a.window) return -1;
    *first = ph == a.b - a.window;
    if (!a.score_rows) return s;
    const int r = __ldg(a.score_rows + s);
    return r >= a.n_score_rows ? -1 : r;  // (the decode records a row out of range)
}

// Records of the rows of one (member, kv head): the G rows of a piece are
// consecutive.
struct PfxPieces {
    long long main, main2, extra;  // first piece, its second stream; row of CTA 0's extra records
    int n, two;                    // pieces, records of each (one per stream); n = 0: none
    int c0, i0, W;                 // set of the first piece; place of its first tile; all places
};

// before, W: the places before the member's group and of all groups.
__device__ __forceinline__ PfxPieces pfx_pieces(const PfxArgs &a, const PfxGroup &g, int mi, int head, int before, int W) {
    PfxPieces p = {};
    if (mi < g.m0 || mi >= g.m0 + g.n || g.tokens == 0) return p;
    const int rt = 1 << a.rt_log, r = (mi - g.m0) << a.G_log, row = r & (rt - 1);
    p.W = W;
    p.i0 = before + (r >> a.rt_log) * (g.lead + g.kts) + g.lead;
    p.c0 = pfx_owner(p.i0, W, a.parts);
    // consecutive sets when each has a place, one tile each otherwise
    p.n = W >= a.parts ? pfx_owner(p.i0 + g.kts - 1, W, a.parts) - p.c0 + 1 : g.kts;
    p.two = a.tc && min(rt, (g.n << a.G_log) - (r - row)) <= rt / 2 ? 2 : 1;  // at most 128 rows: a record per stream
    p.main = pfx_main_row(a, g, head, r);
    p.main2 = p.main + (long long)a.B * a.h_q;
    p.extra = a.extra0 + ((long long)head << a.rt_log) + row;
    return p;
}

// First row of record i in [0, n * two).
__device__ __forceinline__ long long pfx_record(const PfxArgs &a, const PfxPieces &p, int i) {
    const int j = i / p.two, x = i - j * p.two;
    if (j == 0) return x ? p.main2 : p.main;
    const int c = p.W >= a.parts ? p.c0 + j : pfx_owner(p.i0 + j, p.W, a.parts);
    return p.extra + (((long long)c * a.h_kv) << a.rt_log) + (x << (a.rt_log - 1));
}

// Up to these sizes the kernel that joins the records works out where they are.
constexpr int kTailScanB = 512;
constexpr int kTailScanGroups = 256;
__device__ __forceinline__ bool pfx_tail_scans(const PfxArgs &a, int ng) {
    return a.B <= kTailScanB && ng <= kTailScanGroups;
}

// The first CTA's outputs for that kernel beyond (whole CTA).
inline __device__ void pfx_publish(const PfxArgs &a, int ng, const int *pre) {
    if (pfx_tail_scans(a, ng)) return;
    for (int i = threadIdx.x; i <= ng; i += blockDim.x) a.wpre[i] = pre[i];
    for (int s = threadIdx.x; s < a.B; s += blockDim.x) a.place[s] = -1;
    __syncthreads();
    for (int i = threadIdx.x; i < a.B && ng > 0; i += blockDim.x) {
        const PfxGroup g = pfx_group(a, pfx_group_of(a, ng, i));
        if (i < g.m0 || i >= g.m0 + g.n) continue;
        const int s = pfx_member(a, i);
        if (s >= 0) a.place[s] = i;
    }
}

// V consecutive floats through L2.
template <int V>
__device__ __forceinline__ void ld_row(const float *p, float (&v)[V]) {
    if constexpr (V == 4) {
        const float4 w = __ldcg(reinterpret_cast<const float4 *>(p));
        v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
    } else {
        const float2 w = __ldcg(reinterpret_cast<const float2 *>(p));
        v[0] = w.x, v[1] = w.y;
    }
}

// Softmax records of the G rows of a (sequence, kv head) pair joined by SPLIT
// warps of a CTA of four,
//     M = max_j m_j,  L = sum_j 2^(m_j - M) l_j,  acc = sum_j 2^(m_j - M) acc_j.
// A share of the records per warp and, for SPLIT > 1, the warps' results joined in
// shared memory.  Lane i finds record i and its (m, l), 32 at a time; the first
// accumulators are fetched beside the statistics, the others, once it is known which
// records hold anything, U at a time: bound by the latency of these loads.  (With the
// first accumulators behind the statistics: a chain 1 to 2 us longer.)
//   rec(i, ml, acc)  the first row of record i in [0, n): statistics, accumulator
//   put(j, c, y, M, L)  takes V consecutive dims from c of row j (SPLIT 1: V = D/32,
//                       else 1), unnormalised
// Few pairs have many records each, many pairs few: four warps per pair while there are
// at most eight pairs per SM (64 pairs of 17 records, 8 sequences behind 2k tokens: 16 us
// in all, 18 with a warp each; 512 pairs of 20, 64 behind 32k: 59 and 66), else one (2048
// pairs of 7, 256 scored behind 4k: 145 us in all, 159 with four).
constexpr int kJoinWarps = 4;

template <int D, int G, int SPLIT>
struct PfxJoin {
    static constexpr int V = D / 32;
    static constexpr int U = G <= 4 ? 4 : 2;  // records in flight per warp (twice as many: fewer CTAs, 64 x 32k 64 us, not 60)
    struct Smem {
        const float *src[kJoinWarps][32];
        float f[kJoinWarps][32][G];
        float acc[SPLIT > 1 ? SPLIT : 1][G][D];
        float2 ml[SPLIT > 1 ? SPLIT : 1][G];
    };

    template <typename Rec, typename Put>
    static __device__ __forceinline__ void run(Smem &sm, int n, Rec &&rec, Put &&put) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        float M[G], L[G], x[G][V];
#pragma unroll
        for (int j = 0; j < G; ++j) {
            M[j] = -INFINITY;
            L[j] = 0.f;
#pragma unroll
            for (int e = 0; e < V; ++e) x[j][e] = 0.f;
        }
        const int part = SPLIT > 1 ? warp : 0;
        const int n_b = n * part / SPLIT, n_e = n * (part + 1) / SPLIT;
        for (int p0 = n_b; p0 < n_e; p0 += 32) {
            const bool has = p0 + lane < n_e;
            const float2 *ml_p = nullptr;
            const float *acc_p = nullptr;
            if (has) rec(p0 + lane, ml_p, acc_p);
            sm.src[warp][lane] = acc_p;
            float2 ml[G];
#pragma unroll
            for (int j = 0; j < G; ++j) ml[j] = has ? __ldcg(ml_p + j) : make_float2(-INFINITY, 0.f);
            __syncwarp();
            // the first records' accumulators do not wait for the statistics (those of a
            // record that holds nothing are never written: read, and left out)
            float v[U][G][V];
            const int last = min(n_e - p0, 32) - 1;
            auto fetch = [&](int u, int i) {
                const float *src = sm.src[warp][i] + lane * V;
#pragma unroll
                for (int j = 0; j < G; ++j) ld_row<V>(src + j * D, v[u][j]);
            };
#pragma unroll
            for (int u = 0; u < U; ++u) fetch(u, min(u, last));
            // else a stream without a tile (or of weightless tokens only): no accumulator
            // either.  A row whose logits are all NaN has l = NaN: its record counts, and
            // every row decides for itself.
            bool holds = false;
#pragma unroll
            for (int j = 0; j < G; ++j) holds |= !(ml[j].y == 0.f);
            unsigned mask = __ballot_sync(0xFFFFFFFFu, holds);
            if (mask == 0) {
                __syncwarp();
                continue;
            }
#pragma unroll
            for (int j = 0; j < G; ++j) {
                float Mn = fmaxf(M[j], ml[j].x);
#pragma unroll
                for (int o = 16; o; o >>= 1) Mn = fmaxf(Mn, __shfl_xor_sync(0xFFFFFFFFu, Mn, o));
                const float f = ml[j].x == Mn ? 1.f : exp2f(ml[j].x - Mn);  // (both -inf: a sum of 0, or NaN)
                sm.f[warp][lane][j] = f;
                float ls = f * ml[j].y;
#pragma unroll
                for (int o = 16; o; o >>= 1) ls += __shfl_xor_sync(0xFFFFFFFFu, ls, o);
                const float old = M[j] == -INFINITY ? 0.f : exp2f(M[j] - Mn);
                L[j] = L[j] * old + ls;
                M[j] = Mn;
#pragma unroll
                for (int e = 0; e < V; ++e) x[j][e] *= old;
            }
            __syncwarp();
            int at[U];
#pragma unroll
            for (int u = 0; u < U; ++u) at[u] = (mask >> u) & 1 ? u : -1;
            mask &= ~((1u << U) - 1);
            while (true) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (at[u] >= 0) {
#pragma unroll
                        for (int j = 0; j < G; ++j) {
                            const float f = sm.f[warp][at[u]][j];
#pragma unroll
                            for (int e = 0; e < V; ++e) x[j][e] = fmaf(f, v[u][j][e], x[j][e]);
                        }
                    }
                if (mask == 0) break;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    at[u] = __ffs(mask) - 1;  // -1: none left
                    mask &= mask - 1;
                    if (at[u] >= 0) fetch(u, at[u]);
                }
            }
            __syncwarp();
        }
        if constexpr (SPLIT == 1) {
#pragma unroll
            for (int j = 0; j < G; ++j) put(j, lane * V, x[j], M[j], L[j]);
        } else {  // (the pair is the CTA's: every warp is here)
#pragma unroll
            for (int j = 0; j < G; ++j) {
#pragma unroll
                for (int e = 0; e < V; ++e) sm.acc[warp][j][lane * V + e] = x[j][e];
                if (lane == 0) sm.ml[warp][j] = make_float2(M[j], L[j]);
            }
            __syncthreads();
            for (int i = threadIdx.x; i < G * D; i += 32 * SPLIT) {
                const int j = i / D, c = i % D;
                float Mj = -INFINITY, Lj = 0.f, y[1] = {0.f};
#pragma unroll
                for (int w = 0; w < SPLIT; ++w) Mj = fmaxf(Mj, sm.ml[w][j].x);
#pragma unroll
                for (int w = 0; w < SPLIT; ++w) {
                    const float f = sm.ml[w][j].x == -INFINITY ? 0.f : exp2f(sm.ml[w][j].x - Mj);
                    Lj += f * sm.ml[w][j].y;
                    y[0] = fmaf(f, sm.acc[w][j][c], y[0]);
                }
                put(j, c, y, Mj, Lj);
            }
        }
    }
};

// One score: written, or added to what the window's earlier steps left.  Every score
// has one thread, so that the order of the additions is that of the steps.
__device__ __forceinline__ void pfx_put_score(float *p, float v, bool on, bool write) {
    st_if(p, v, on && write);
    add_if(p, v, on && !write);
}

// Window score of the tokens behind the prefixes, from the decode's logits and the
// final statistics: S[t] (+)= (1/w) max_{h in group} 2^(x_ht - m_h) / l_h, written
// instead of added at the first window row and for the newest token.  A share of
// the units per CTA, a thread per (token, kv head) of a unit (at most 256 of them:
// the units' bytes bound it); consecutive threads take consecutive tokens, and a
// thread's kv head stays, so its statistics are read when the sequence changes.
template <int G, int THREADS>
__device__ __forceinline__ void pfx_own_scores(const PfxArgs &a, int tid) {
    const int U = __ldcg(a.n_units);
    const int u0 = (int)((long long)U * blockIdx.x / gridDim.x), u1 = (int)((long long)U * (blockIdx.x + 1) / gridDim.x);
    const int items = a.h_kv << a.unit_log, per = THREADS / items;
    const int q = tid / items, kvh = (tid >> a.unit_log) % a.h_kv, tl = tid & ((1 << a.unit_log) - 1);
    const float inv_w = 1.f / (float)a.window;
    constexpr int K = G <= 4 ? 8 : 4;  // units in flight per thread
    int last = -1;
    float *row = nullptr;
    float c[G];
#pragma unroll
    for (int j = 0; j < G; ++j) c[j] = INFINITY;
    for (int ub = u0 + q; ub < u1; ub += K * per) {
        int4 info[K];
        float x[K][G];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int u = ub + k * per;
            info[k] = u < u1 ? __ldcg(a.units + u) : make_int4(0, 0, 0, 0);
            // (logits of units that are not on a window step hold anything)
            const float *lg = a.logits + (((size_t)min(u, u1 - 1) << a.unit_log) + tl) * a.h_q + kvh * G;
            if constexpr (G >= 4) {
#pragma unroll
                for (int j = 0; j < G; j += 4)
                    *reinterpret_cast<float4 *>(&x[k][j]) = __ldcg(reinterpret_cast<const float4 *>(lg + j));
            } else {
#pragma unroll
                for (int j = 0; j < G; ++j) x[k][j] = __ldcg(lg + j);
            }
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int tok = info[k].y + tl;
            const bool on = (info[k].w & 1) && tok < info[k].z;
            if (on && info[k].x != last) {
                last = info[k].x;
#pragma unroll
                for (int j = 0; j < G; ++j) c[j] = __ldcg(a.stats + (size_t)last * a.h_q + kvh * G + j);
                // the row was checked by the decode (a unit without one carries no window flag)
                const int r = a.score_rows ? __ldg(a.score_rows + last) : last;
                const int first_tok = min(__ldg(a.seq_lens + last), a.stride * a.b) - info[k].z;
                row = a.score + ((size_t)r * a.h_kv + kvh) * a.score_stride + first_tok;
            }
            float e = x[k][0] - c[0];
#pragma unroll
            for (int j = 1; j < G; ++j) e = fmaxf(e, x[k][j] - c[j]);
            pfx_put_score(row + tok, exp2f(e) * inv_w, on, (info[k].w & 2) || tok == info[k].z - 1);
        }
    }
}

// Host: four warps per pair while the pairs' CTAs are resident at once.
inline bool pfx_join_split(const PfxArgs &a) { return (long long)a.B * a.h_kv <= 8LL * a.parts * a.h_kv; }

}  // namespace zp
