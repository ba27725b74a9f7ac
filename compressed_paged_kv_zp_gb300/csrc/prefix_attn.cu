// prefix_attn.cu -- decode attention of a batch whose sequences share prefixes:
// the shared part computed once per group for all its members.
//
// For a group of n sequences that share p prefix tokens, the G query rows of a
// kv head of every member form one matrix of n*G rows, and its attention to the
// shared keys and values is a dense product:
//     x = log2(e)/sqrt(d) Q K^T,  m_r = max_t x_rt,  l_r = sum_t 2^(x_rt - m_r),
//     acc_r = sum_t 2^(x_rt - m_r) v_t.
// (m, l, acc) of every (sequence, q head) and the decode's of the sequence's other
// tokens (decode_attn_prefix.cu) join to the softmax over all tokens, so the shared
// keys and values are read once per group instead of once per sequence.  With the
// window score, the final (m, l) give a second pass over the shared keys for the
// sequences on a window step, and over the decode's logits:
//     S[t] (+)= (1/w) max_{h in group} 2^(x_ht - m_h) / l_h.
// Chain of launches: the prefix kernel; the decode, which needs nothing of it and
// follows without a gap; the kernel that joins the records; the score.  8 sequences
// behind 2k tokens 16 us, 64 behind 32k 60, scored 256 behind 4k 147 (bf16, 32 q and 8
// kv heads of 128).  With the decode starting from the joined prefix instead, and its
// own cooperative merge and score, the first two took 24 and 73.
//
// Work: an item is (group, tile of query rows), its length the group's tiles of
// prefix tokens.  The tiles of all items are concatenated and every set of h_kv
// CTAs takes an equal contiguous range (as the decode does with its units), one
// kv head per CTA, so any mix of group sizes and prefix lengths fills the GPU
// and the CTAs of a set read the heads of the same token rows at the same time.
// The first piece of an item goes to its rows' place in the main records, a
// piece that begins inside an item (at most one per CTA) to the CTA's extra
// records.
#include <math.h>

#include "prefix_tc.h"

namespace zp {
namespace {

constexpr int kPfxThreads = 256;
constexpr int kPfxRows = 64;    // query rows per item
constexpr int kPfxTokens = 64;  // prefix tokens per tile

// Four consecutive elements.
__device__ __forceinline__ void load_vec(const float *p, float *o) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    o[0] = v.x, o[1] = v.y, o[2] = v.z, o[3] = v.w;
}

// ===========================================================================
// CUDA-core kernels (fp32 caches; bf16 caches: prefix_tc.cu).
// 64 query rows x 64 prefix tokens per tile, everything in fp32 in shared
// memory; a thread holds 4 rows x 4 tokens of the logits and 4 rows x d/16 dims
// of the accumulator, and the 16 threads of a row (a half-warp) share its
// softmax statistics by shuffles: eight 16-byte loads per 64 FMAs.  The next tile waits
// in registers while one is computed.  With few tiles per CTA bound by latency, the plan's
// scan, the queries and the first tile one after another: 61 sequences in 7 groups behind
// 672 tokens, 16 q and 4 kv heads of 64, two tiles per CTA, 10 us and scored in all 40 us
// (4.4 TFLOP/s); of this kernel's cycles 28 % issue and 12 % use the fp32 pipe.
template <int D>
struct PfxSmem {
    float q[kPfxRows][D + 4];
    float k[kPfxTokens][D + 4];
    float v[kPfxTokens][D];
    float p[kPfxRows][kPfxTokens + 4];
};

// Query rows [r0, r0 + 64) of the group into shared memory, zero beyond the last.
template <int D, int G>
__device__ void pfx_load_q(const PfxArgs &a, const PfxGroup &g, int head, int r0, PfxSmem<D> &sm) {
    constexpr int V = 4;
    for (int i = threadIdx.x; i < kPfxRows * (D / V); i += kPfxThreads) {
        const int r = i / (D / V), c = (i % (D / V)) * V;
        float x[V];
#pragma unroll
        for (int e = 0; e < V; ++e) x[e] = 0.f;
        if (r0 + r < g.n * G) {
            const int s = pfx_member(a, g.m0 + (r0 + r) / G);
            if (s >= 0)
                load_vec(static_cast<const float *>(a.q) + ((size_t)s * a.h_q + head * G + (r0 + r) % G) * D + c, x);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) sm.q[r][c + e] = x[e] * a.qscale;
    }
}

// 64 prefix tokens from t0 (zero beyond the prefix and for bad blocks): fetched
// into registers while the tile before is computed, then put in shared memory.
template <int D, bool WITH_V>
struct PfxFetch {
    static constexpr int N = kPfxTokens * (D / 4) / kPfxThreads;
    float4 k[N], v[WITH_V ? N : 1];

    __device__ __forceinline__ void load(const PfxArgs &a, const PfxGroup &g, const int32_t *row, int head, int t0) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int i = n * kPfxThreads + threadIdx.x, t = i / (D / 4), c = (i % (D / 4)) * 4;
            k[n] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (WITH_V) v[n] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (t0 + t < g.tokens) {
                const long long slot = pfx_slot(a, row, t0 + t);
                if (slot >= 0) {
                    const size_t at = ((size_t)slot * a.h_kv + head) * D + c;
                    k[n] = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(a.k) + at));
                    if (WITH_V) v[n] = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(a.v) + at));
                }
            }
        }
    }
    __device__ __forceinline__ void store(PfxSmem<D> &sm) const {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int i = n * kPfxThreads + threadIdx.x, t = i / (D / 4), c = (i % (D / 4)) * 4;
            *reinterpret_cast<float4 *>(&sm.k[t][c]) = k[n];
            if (WITH_V) *reinterpret_cast<float4 *>(&sm.v[t][c]) = v[n];
        }
    }
};

// Logits of rows ty*4 + i, tokens tx + 16 j (log2 units).
template <int D>
__device__ __forceinline__ void pfx_logits(const PfxSmem<D> &sm, int ty, int tx, float (&x)[4][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = 0.f;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
        float4 qv[4], kv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) qv[i] = *reinterpret_cast<const float4 *>(&sm.q[ty * 4 + i][c]);
#pragma unroll
        for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4 *>(&sm.k[tx + 16 * j][c]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[i][j] = fmaf(qv[i].x, kv[j].x, x[i][j]);
                x[i][j] = fmaf(qv[i].y, kv[j].y, x[i][j]);
                x[i][j] = fmaf(qv[i].z, kv[j].z, x[i][j]);
                x[i][j] = fmaf(qv[i].w, kv[j].w, x[i][j]);
            }
    }
}

template <int D, int G>
__global__ void __launch_bounds__(kPfxThreads) prefix_part_kernel(const PfxArgs a) {
    extern __shared__ __align__(16) unsigned char pfx_raw[];
    PfxSmem<D> &sm = *reinterpret_cast<PfxSmem<D> *>(pfx_raw);
    int *pre = reinterpret_cast<int *>(pfx_raw + sizeof(PfxSmem<D>));
    constexpr int DV = D / 64;  // float4 groups of dims per thread
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int ng = pfx_groups(a);
    const int W = pfx_scan(a, ng, pre);
    pdl_trigger();
    if (blockIdx.x == 0) pfx_publish(a, ng, pre);
    const int head = blockIdx.x % a.h_kv, set = blockIdx.x / a.h_kv;
    const int w0 = pfx_start(set, W, a.parts), w1 = pfx_start(set + 1, W, a.parts);
    for (int w = w0; w < w1;) {
        const PfxSeg seg = pfx_segment(a, pre, ng, w, w1);
        const PfxGroup &g = seg.g;
        const int t_b = seg.t_b, t_e = seg.t_e, r0 = seg.item * kPfxRows;
        w = seg.w_e;
        if (t_b == t_e) continue;
        const int32_t *row = pfx_row(a, g);
        __syncthreads();  // the last segment's reads of shared memory
        pfx_load_q<D, G>(a, g, head, r0, sm);
        float m[4], l[4], acc[4][4 * DV];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int e = 0; e < 4 * DV; ++e) acc[i][e] = 0.f;
        }
        PfxFetch<D, true> next;
        next.load(a, g, row, head, t_b * kPfxTokens);
        const bool live = r0 + (ty & ~1) * 4 < g.n * G;  // the warp has a query row
        for (int t = t_b; t < t_e; ++t) {
            const int t0 = t * kPfxTokens;
            __syncthreads();
            next.store(sm);
            __syncthreads();
            if (t + 1 < t_e) next.load(a, g, row, head, t0 + kPfxTokens);
            if (!live) continue;
            float x[4][4];
            pfx_logits<D>(sm, ty, tx, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float mx = m[i];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (t0 + tx + 16 * j >= g.tokens) x[i][j] = -INFINITY;
                    mx = fmaxf(mx, x[i][j]);
                }
#pragma unroll
                for (int o = 1; o < 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
                // (the tile's first token is in the prefix: the maximum is that of at least one logit)
                const float al = mx == -INFINITY ? 1.f : exp2f(m[i] - mx);
                m[i] = mx;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p = x[i][j] == -INFINITY ? 0.f : exp2f(x[i][j] - mx);
                    sum += p;
                    sm.p[ty * 4 + i][tx + 16 * j] = p;
                }
                l[i] = l[i] * al + sum;  // this thread's tokens only; joined at the end
#pragma unroll
                for (int e = 0; e < 4 * DV; ++e) acc[i][e] *= al;
            }
            __syncwarp();  // the rows of a half-warp's p are its own
#pragma unroll 2
            for (int t4 = 0; t4 < kPfxTokens; t4 += 4) {
                float4 pv[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) pv[i] = *reinterpret_cast<const float4 *>(&sm.p[ty * 4 + i][t4]);
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int dv = 0; dv < DV; ++dv) {
                        const float4 vv = *reinterpret_cast<const float4 *>(&sm.v[t4 + u][dv * 64 + tx * 4]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float p = u == 0 ? pv[i].x : (u == 1 ? pv[i].y : (u == 2 ? pv[i].z : pv[i].w));
                            acc[i][4 * dv] = fmaf(p, vv.x, acc[i][4 * dv]);
                            acc[i][4 * dv + 1] = fmaf(p, vv.y, acc[i][4 * dv + 1]);
                            acc[i][4 * dv + 2] = fmaf(p, vv.z, acc[i][4 * dv + 2]);
                            acc[i][4 * dv + 3] = fmaf(p, vv.w, acc[i][4 * dv + 3]);
                        }
                    }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], o);
            const int r = r0 + ty * 4 + i;
            if (r < g.n * G) {
                const long long at = t_b == 0 ? pfx_main_row(a, g, head, r)
                                              : a.extra0 + (long long)blockIdx.x * kPfxRows + ty * 4 + i;
                if (tx == 0) a.rec_ml[at] = make_float2(m[i], l[i]);
#pragma unroll
                for (int dv = 0; dv < DV; ++dv)
                    *reinterpret_cast<float4 *>(a.rec_acc + at * D + dv * 64 + tx * 4) =
                        make_float4(acc[i][4 * dv], acc[i][4 * dv + 1], acc[i][4 * dv + 2], acc[i][4 * dv + 3]);
            }
        }
    }
}

// Window score of the prefix tokens from the final statistics: the logits again,
// the maximum of x - (m + log2 l) over the q heads of the kv head, one
// exponential per (sequence, kv head, token).  The first tile's logits do not wait for
// the statistics (40 us where all of it waits: 45).
template <int D, int G>
__global__ void __launch_bounds__(kPfxThreads) prefix_score_kernel(const PfxArgs a) {
    extern __shared__ __align__(16) unsigned char pfx_raw[];
    PfxSmem<D> &sm = *reinterpret_cast<PfxSmem<D> *>(pfx_raw);
    int *pre = reinterpret_cast<int *>(pfx_raw + sizeof(PfxSmem<D>));
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int ng = pfx_groups(a);
    const int W = pfx_scan(a, ng, pre);
    const int head = blockIdx.x % a.h_kv, set = blockIdx.x / a.h_kv;
    const int w0 = pfx_start(set, W, a.parts), w1 = pfx_start(set + 1, W, a.parts);
    bool waited = false;
    const float inv_w = 1.f / (float)a.window;
    for (int w = w0; w < w1;) {
        const PfxSeg seg = pfx_segment(a, pre, ng, w, w1);
        const PfxGroup &g = seg.g;
        const int t_b = seg.t_b, t_e = seg.t_e, r0 = seg.item * kPfxRows;
        w = seg.w_e;
        if (t_b == t_e) continue;
        const int32_t *row = pfx_row(a, g);
        __syncthreads();
        pfx_load_q<D, G>(a, g, head, r0, sm);
        // score row of this thread's rows, and where their c = m + log2 l stands
        float c[4];
        const float *c_at[4];
        int srow[4];
        bool first[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = r0 + ty * 4 + i;
            c[i] = INFINITY;
            c_at[i] = a.stats;
            srow[i] = -1;
            first[i] = false;
            if (r < g.n * G) {
                const int s = pfx_member(a, g.m0 + r / G);
                if (s >= 0) {
                    srow[i] = pfx_score_row(a, s, &first[i]);
                    c_at[i] = a.stats + (size_t)s * a.h_q + head * G + r % G;
                }
            }
        }
        PfxFetch<D, false> next;
        next.load(a, g, row, head, t_b * kPfxTokens);
        const bool live = r0 + (ty & ~1) * 4 < g.n * G;  // the warp has a query row
        for (int t = t_b; t < t_e; ++t) {
            const int t0 = t * kPfxTokens;
            __syncthreads();
            next.store(sm);
            __syncthreads();
            if (t + 1 < t_e) next.load(a, g, row, head, t0 + kPfxTokens);
            if (!live) continue;
            // a score per four rows (the thread's are of one entry), for G = 8 per eight
            const bool scores = srow[0] >= 0 && !(G == 8 && (ty & 1));
            float *at = a.score + ((size_t)max(srow[0], 0) * a.h_kv + head) * a.score_stride + t0 + tx;
            float x[4][4];
            pfx_logits<D>(sm, ty, tx, x);
            if (t == t_b) {  // the final statistics: the first logits are formed before they are
                if (!waited) pdl_wait();
                waited = true;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (srow[i] >= 0) c[i] = __ldcg(c_at[i]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float e[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) e[i] = x[i][j] - c[i];
                // maximum over the group's rows: four inside the thread, for G = 8 with the
                // other half-warp's (the next four rows)
                e[0] = fmaxf(fmaxf(e[0], e[1]), fmaxf(e[2], e[3]));
                if constexpr (G == 8) e[0] = fmaxf(e[0], __shfl_xor_sync(0xFFFFFFFFu, e[0], 16));
                pfx_put_score(at + 16 * j, exp2f(e[0]) * inv_w, scores && t0 + tx + 16 * j < g.tokens, first[0]);
            }
        }
    }
    if (!waited) pdl_wait();
    pfx_own_scores<G, kPfxThreads>(a, tid);
}

struct PfxPlan {
    bool tc;
    int rt, kt, parts;
    long long extra0;
    size_t off_wpre, off_place, off_rml, off_racc, off_wml, off_wacc, total;
};

zp_status pfx_plan(const zp_cache_desc *D, int B, const DeviceInfo &dev, PfxPlan *p) {
    const int d = D->head_dim, G = D->h_q / D->h_kv;
    if (!(d == 64 || d == 128)) return fail(ZP_ERR_SHAPE, "prefix_decode: head_dim %d not in {64,128}", d);
    if (!(G == 1 || G == 2 || G == 4 || G == 8)) return fail(ZP_ERR_SHAPE, "prefix_decode: group size %d", G);
    if (B > kPfxMaxB) return fail(ZP_ERR_SHAPE, "prefix_decode: B %d > %d", B, kPfxMaxB);
    p->tc = D->dtype == ZP_BF16;
    p->rt = p->tc ? kPtRows : kPfxRows;
    p->kt = p->tc ? 128 : kPfxTokens;
    p->parts = dev.sm_count / D->h_kv;
    if (p->parts < 1) return fail(ZP_ERR_SHAPE, "prefix_decode: h_kv %d above %d", D->h_kv, dev.sm_count);
    const size_t rows = (size_t)B * D->h_q;
    p->extra0 = (long long)(p->tc ? 2 * rows : rows);
    const size_t recs = (size_t)p->extra0 + (size_t)p->parts * D->h_kv * p->rt;
    size_t off = 0;
    p->off_wpre = off;
    off = align_up(off + (size_t)(B + 1) * 4, 256);
    p->off_place = off;
    off = align_up(off + (size_t)B * 4, 256);
    p->off_rml = off;
    off = align_up(off + recs * 8, 256);
    p->off_racc = off;
    off = align_up(off + recs * d * 4, 256);
    p->off_wml = off;
    off = align_up(off + rows * 8, 256);
    p->off_wacc = off;
    off = align_up(off + rows * d * 4, 256);
    p->total = off;
    return ZP_OK;
}

template <int D, int G>
zp_status launch_part(const PfxArgs &a, cudaStream_t st) {
    const size_t smem = sizeof(PfxSmem<D>) + (size_t)(a.B + 1) * 4;
    zp_status rc = set_max_dynamic_smem(reinterpret_cast<const void *>(prefix_part_kernel<D, G>), smem,
                                        "prefix_decode: shared-memory attribute");
    if (rc != ZP_OK) return rc;
    prefix_part_kernel<D, G><<<a.parts * a.h_kv, kPfxThreads, smem, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "prefix_decode: prefix kernel launch");
    return ZP_OK;
}

template <int D, int G>
zp_status launch_score(const PfxArgs &a, cudaStream_t st) {
    const size_t smem = sizeof(PfxSmem<D>) + (size_t)(a.B + 1) * 4;
    zp_status rc = set_max_dynamic_smem(reinterpret_cast<const void *>(prefix_score_kernel<D, G>), smem,
                                        "prefix_decode: shared-memory attribute");
    if (rc != ZP_OK) return rc;
    const cudaError_t e = launch_dependent(prefix_score_kernel<D, G>, dim3(a.parts * a.h_kv), dim3(kPfxThreads), smem, st, a);
    if (e != cudaSuccess) return cuda_fail(e, "prefix_decode: score kernel launch");
    return ZP_OK;
}

// fp32 caches: the kernel of the head dimension and group size (4 or 8, as the decode's).
template <int D>
zp_status launch_part_f32(const PfxArgs &a, int G, cudaStream_t st) {
    if (G == 4) return launch_part<D, 4>(a, st);
    return launch_part<D, 8>(a, st);
}
template <int D>
zp_status launch_score_f32(const PfxArgs &a, int G, cudaStream_t st) {
    if (G == 4) return launch_score<D, 4>(a, st);
    return launch_score<D, 8>(a, st);
}

}  // namespace
}  // namespace zp

using namespace zp;

extern "C" size_t zp_prefix_decode_workspace_size(const zp_cache_desc *D, int32_t B, int32_t table_stride) {
    if (check_desc(D) != ZP_OK || B < 0 || table_stride < 0) return 0;
    const size_t dec = zp_decode_workspace_size(D, B, table_stride);
    DeviceInfo dev;
    PfxPlan p;
    if (dec == 0 || device_info(&dev) != ZP_OK || pfx_plan(D, B, dev, &p) != ZP_OK) return 0;
    return align_up(dec, 256) + p.total;
}

extern "C" zp_status zp_prefix_decode_attn(const zp_cache_desc *D, const void *q, const void *k_cache,
                                           const void *v_cache, const int32_t *block_table, int32_t table_stride,
                                           const int32_t *seq_lens, int32_t B, const zp_prefix_groups *plan, void *out,
                                           float *score_accum, const int32_t *score_rows, int32_t n_score_rows,
                                           int32_t window, void *workspace, size_t workspace_bytes, void *stream) {
    zp_status rc = check_desc(D);
    if (rc != ZP_OK) return rc;
    if (B < 0 || table_stride < 0) return fail(ZP_ERR_INVALID_ARG, "prefix_decode: B or table_stride negative");
    if (B == 0) return ok();
    if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !out || !workspace || !plan || !plan->prefix_lens || !plan->n_groups ||
        !plan->group_start || !plan->members || !plan->group_blocks)
        return fail(ZP_ERR_INVALID_ARG, "prefix_decode: NULL buffer");
    if (table_stride < 1) return fail(ZP_ERR_INVALID_ARG, "prefix_decode: table_stride < 1");
    if (score_accum && (window < 1 || window > D->block_size))
        return fail(ZP_ERR_INVALID_ARG, "prefix_decode: window %d outside [1, b=%d]", window, D->block_size);
    if (score_accum && score_rows && n_score_rows < 1)
        return fail(ZP_ERR_INVALID_ARG, "prefix_decode: a slot map needs n_score_rows >= 1");
    const uintptr_t al = (uintptr_t)q | (uintptr_t)k_cache | (uintptr_t)v_cache | (uintptr_t)out |
                         (uintptr_t)score_accum | (uintptr_t)workspace;
    if (al % 16) return fail(ZP_ERR_INVALID_ARG, "prefix_decode: buffers must be 16-byte aligned");
    // the score forms the prefix's logits again, from the queries, when the outputs are written
    const uintptr_t rows = (uintptr_t)B * D->h_q * D->head_dim * elem_bytes(D->dtype);
    if (score_accum && (uintptr_t)q < (uintptr_t)out + rows && (uintptr_t)out < (uintptr_t)q + rows)
        return fail(ZP_ERR_INVALID_ARG, "prefix_decode: out overlaps q in a scored call");
    const int G = D->h_q / D->h_kv;
    // tile counts are 32-bit: query rows * tiles of a table row bounds them
    if (((double)B * G) * ((double)table_stride * D->block_size / kPfxTokens + 1) > 2147483647.0 ||
        (long long)table_stride * D->block_size > INT32_MAX)
        return fail(ZP_ERR_SHAPE, "prefix_decode: B=%d rows of %d blocks", B, table_stride);
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != ZP_OK) return rc;
    PfxPlan p;
    rc = pfx_plan(D, B, dev, &p);
    if (rc != ZP_OK) return rc;
    const size_t dec = zp_decode_workspace_size(D, B, table_stride);
    if (dec == 0) return fail(ZP_ERR_SHAPE, "prefix_decode: %s", zp_last_error());
    if (workspace_bytes < align_up(dec, 256) + p.total)
        return fail(ZP_ERR_CAPACITY, "prefix_decode: workspace %zu < %zu bytes", workspace_bytes,
                    align_up(dec, 256) + p.total);
    unsigned char *ws = static_cast<unsigned char *>(workspace) + align_up(dec, 256);
    PfxArgs a = {};
    a.q = q;
    a.k = k_cache;
    a.v = v_cache;
    a.table = block_table;
    a.stride = table_stride;
    a.seq_lens = seq_lens;
    a.B = B;
    a.h_q = D->h_q;
    a.h_kv = D->h_kv;
    a.b = D->block_size;
    a.b_log = __builtin_ctz((unsigned)D->block_size);  // (a power of two: the decode's plan checked it)
    a.G = G;
    a.G_log = __builtin_ctz((unsigned)G);
    a.n_total = D->n_total_blocks;
    a.prefix = plan->prefix_lens;
    a.n_groups = plan->n_groups;
    a.group_start = plan->group_start;
    a.members = plan->members;
    a.group_blocks = plan->group_blocks;
    a.rt_log = __builtin_ctz((unsigned)p.rt);
    a.kt_log = __builtin_ctz((unsigned)p.kt);
    a.parts = p.parts;
    a.extra0 = p.extra0;
    a.tc = p.tc;
    a.qscale = (float)(1.4426950408889634 / sqrt((double)D->head_dim));
    a.wpre = reinterpret_cast<int *>(ws + p.off_wpre);
    a.rec_acc = reinterpret_cast<float *>(ws + p.off_racc);
    a.rec_ml = reinterpret_cast<float2 *>(ws + p.off_rml);
    a.place = reinterpret_cast<int *>(ws + p.off_place);
    a.whole_acc = reinterpret_cast<float *>(ws + p.off_wacc);
    a.whole_ml = reinterpret_cast<float2 *>(ws + p.off_wml);
    a.score = score_accum;
    a.score_stride = (long long)table_stride * D->block_size;
    a.score_rows = score_accum ? score_rows : nullptr;
    a.n_score_rows = n_score_rows;
    a.window = window;
    a.err = dev.error_word;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int d = D->head_dim;
    if (p.tc) rc = prefix_part_tc(a, d, st);
    else rc = d == 64 ? launch_part_f32<64>(a, G, st) : launch_part_f32<128>(a, G, st);
    if (rc != ZP_OK) return rc;
    rc = decode_after_prefix(D, q, k_cache, v_cache, block_table, table_stride, seq_lens, B, out, score_accum, score_rows,
                             n_score_rows, window, a, workspace, dec, stream);
    if (rc != ZP_OK) return rc;
    if (score_accum) {
        if (p.tc) rc = prefix_score_tc(a, d, st);
        else rc = d == 64 ? launch_score_f32<64>(a, G, st) : launch_score_f32<128>(a, G, st);
        if (rc != ZP_OK) return rc;
    }
    return ok();
}
