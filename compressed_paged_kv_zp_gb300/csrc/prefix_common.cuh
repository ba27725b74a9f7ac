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
    int B, h_q, h_kv, b, n_total;
    // the plan
    const int32_t *n_groups, *group_start, *members, *group_blocks;
    int rt, kt;          // rows per item, tokens per tile
    int parts;           // sets of CTAs (split of the tiles); a set has a CTA per kv head
    float qscale;        // log2(e) / sqrt(d)
    int *wpre;           // [B+1] tiles before each group
    int32_t *prefix;     // [B] prefix tokens of every batch entry, 0 = none
    float *rec_acc;      // [extra0 + parts*rt][d] pieces: main records, then extra records
    float2 *rec_ml;      // same rows
    long long extra0;    // first extra record: B*h_q, twice that on the tensor cores (second streams);
                         // then rt rows per CTA (set * h_kv + head)
    int tc;              // tensor-core kernels: 256 rows x 128 tokens, two streams
    float *init_acc;     // [B][h_q][d]
    float2 *init_ml;     // [B][h_q]
    // score
    float *score;
    long long score_stride;
    const int32_t *score_rows;
    int n_score_rows, window;
    const float2 *stats;  // [B][h_q] final (max, sum)
    unsigned *err;
};

// Group g of the plan, with every index the plan gives bounded.
struct PfxGroup {
    int m0, n;    // first member, members
    int tokens;   // prefix tokens
    int rts, kts; // row tiles, token tiles
};

__device__ __forceinline__ int pfx_groups(const PfxArgs &a) { return min(max(__ldg(a.n_groups), 0), a.B); }

__device__ __forceinline__ PfxGroup pfx_group(const PfxArgs &a, int g) {
    PfxGroup r;
    r.m0 = min(max(__ldg(a.group_start + g), 0), a.B);
    r.n = min(max(__ldg(a.group_start + g + 1), r.m0), a.B) - r.m0;
    r.tokens = min(max(__ldg(a.group_blocks + g), 0), a.stride) * a.b;
    r.rts = (r.n * (a.h_q / a.h_kv) + a.rt - 1) / a.rt;
    r.kts = (r.tokens + a.kt - 1) / a.kt;
    return r;
}

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

// Tiles before each group (whole CTA; pre: n_groups + 1 ints of shared memory);
// returns the total.
inline __device__ int pfx_scan(const PfxArgs &a, int ng, int *pre) {
    for (int i = threadIdx.x; i < ng; i += blockDim.x) {
        const PfxGroup g = pfx_group(a, i);
        pre[i] = g.rts * g.kts;
    }
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

// Row of the main records: rows of a group are (kv head, member, q head of the
// group), after the rows of the members before it.
__device__ __forceinline__ long long pfx_main_row(const PfxArgs &a, const PfxGroup &g, int head, int r) {
    return (long long)g.m0 * a.h_q + (long long)head * g.n * (a.h_q / a.h_kv) + r;
}

// Physical row (block * b + slot) of token t of the group's prefix, by its first
// member's table row; -1 for a bad block id (recorded).
__device__ __forceinline__ long long pfx_slot(const PfxArgs &a, const int32_t *row, int t) {
    const int blk = __ldg(row + t / a.b);
    if (blk < 0 || blk >= a.n_total) {
        record_error(a.err, ZP_ERR_DEVICE, 0x143);
        return -1;
    }
    return (long long)blk * a.b + t % a.b;
}

// The table row every member's prefix agrees with: the first member's.
__device__ __forceinline__ const int32_t *pfx_row(const PfxArgs &a, const PfxGroup &g) {
    const int s = pfx_member(a, g.m0);
    return a.table + (size_t)(s < 0 ? 0 : s) * a.stride;
}

// Row of the score that batch entry s adds to in this step, -1: none (no prefix,
// not on a window step, no score row).  first: the window's first row, written.
__device__ __forceinline__ int pfx_score_row(const PfxArgs &a, int s, bool *first) {
    const int L = min(__ldg(a.seq_lens + s), a.stride * a.b);
    const int p = a.prefix[s];
    *first = false;
    if (p <= 0 || p >= L) return -1;
    const int ph = (L - 1) % a.b;
    if (ph < a.b - a.window) return -1;
    *first = ph == a.b - a.window;
    if (!a.score_rows) return s;
    const int r = __ldg(a.score_rows + s);
    return r >= a.n_score_rows ? -1 : r;  // (the decode records a row out of range)
}

// The first CTA's outputs for the kernels that follow: the tiles before each
// group and the prefix tokens of every batch entry (whole CTA).
inline __device__ void pfx_publish(const PfxArgs &a, int ng, const int *pre) {
    for (int i = threadIdx.x; i <= ng; i += blockDim.x) a.wpre[i] = pre[i];
    for (int s = threadIdx.x; s < a.B; s += blockDim.x) a.prefix[s] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < a.B && ng > 0; i += blockDim.x) {
        const PfxGroup g = pfx_group(a, pfx_group_of(a, ng, i));
        if (i < g.m0 || i >= g.m0 + g.n) continue;
        const int s = pfx_member(a, i);
        if (s >= 0) a.prefix[s] = g.tokens;
    }
}

}  // namespace zp
