// prefix_plan.cu -- groups of sequences that share their leading blocks, found
// on the GPU from the block table.
//
// Sequence s with L_s tokens may share its first u_s = (L_s - 1) / b blocks
// (never the one that holds the newest token).  Sequences with u_s >= 1 and the
// same first block form a class; its leader is the one with the largest u
// (lowest index on ties); lcp_s is the number of leading entries that s and
// the leader have in common, at most min(u_s, u_leader).  The class shares the
// p blocks that save the most reads,
//     p = argmax over its lcp values of p * (#{j : lcp_j >= p} - 1),
// the longer p on ties, among the members with lcp >= p.  A class with fewer
// than min_members (>= 2) such members, or p < min_blocks, gives no group.
//
// One cluster of CTAs, a slice of the batch per CTA: a shared-memory hash of the
// first blocks finds the leaders (each CTA builds it from all B first entries),
// a warp compares table rows, lcp and counts are exchanged through distributed
// shared memory (a sequence is counted against its own class only, whose members
// are listed together), and the first CTA numbers the groups.  Bound by
// latency (four cluster barriers and the gather of the first column); the rows
// are read only up to their first difference.  256 entries behind a prefix of 64
// blocks: 11.7 us; 2048 behind 16 prefixes of up to 256: 28.8 us, of which hashing 3.4,
// the rows 7.5, counting and ranking 5 (the launch, the gather, the barriers and the first
// CTA's numbering were not timed apart).
#include <cooperative_groups.h>

#include "zp_common.cuh"

namespace zp {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanMaxB = 4096;
constexpr int kPlanCluster = 8;
constexpr int kPlanHash = 8192;  // slots, twice the largest batch

struct PlanArgs {
    const int32_t *table;
    int stride;
    const int32_t *seq_lens;
    int B, b, n_total;
    int min_blocks, min_members;
    int32_t *prefix_lens, *n_groups, *group_start, *members, *group_blocks;
};

// Shared memory of one CTA.
static_assert(kPlanHash >= 2 * kPlanMaxB && kPlanMaxB == 1 << 12, "arrays over the hash; 12 bits of an index");
struct PlanSmem {
    union {
        int key[kPlanHash];              // first block id, -1 = free
        struct {                         // once the leaders are known:
            unsigned gain[kPlanMaxB];    // by leader: most blocks saved
            int shared[kPlanMaxB];       // by leader: the longest lcp that saves them
        };
    };
    union {
        struct {
            int most[kPlanHash];         // largest u of the class
            int lead[kPlanHash];         // its leader: the lowest index with that u
        };
        struct {                         // once the leaders are known, by leader:
            int cls_n[kPlanMaxB];        // sequences of the class
            int cls_at[kPlanMaxB];       // its first place in seg
            unsigned seg[kPlanMaxB];     // the classes one after another: (lcp << 12) | index
        };
    };
    int leader[kPlanMaxB];               // leader of each sequence, -1 = no class
    int lcp[kPlanMaxB];
    alignas(16) int aux[kPlanMaxB];      // members with at least this lcp, then the rank inside the group
    int gid[kPlanMaxB];                  // by leader: lowest member, then group number
    int size[kPlanMaxB];                 // by leader: members
    int full[kPlanMaxB];                 // blocks before the newest token's
    alignas(4) unsigned char member[kPlanMaxB];
    int warp_sums[32];
    int total;
};

__device__ __forceinline__ int plan_scan(int x, PlanSmem &sm) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int v = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += y;
    }
    if (lane == 31) sm.warp_sums[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int w = sm.warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, w, o);
            if (lane >= o) w += y;
        }
        sm.warp_sums[lane] = w;
    }
    __syncthreads();
    const int before = warp ? sm.warp_sums[warp - 1] : 0;
    if (threadIdx.x == 0) sm.total = sm.warp_sums[31];
    __syncthreads();
    return before + v - x;
}

__device__ __forceinline__ unsigned plan_hash(int id) { return ((unsigned)id * 2654435761u) >> 19; }  // 13 bits

__device__ __forceinline__ int plan_full(const PlanArgs &a, int s) {
    int L = a.seq_lens[s];
    if (L > a.stride * a.b) L = a.stride * a.b;
    return L > 0 ? (L - 1) / a.b : 0;
}

constexpr int kWarps = kPlanThreads / 32;

// lcp of sequences [e0, e1) with their leaders, written to every CTA: EACH rows per
// warp at a time, 128 entries of each, all loads in flight.  Bound by the
// instructions per entry, so a column beyond the row's limit reads the last one
// again instead of being tested, and a chunk is searched only if it differs.
template <int EACH>
__device__ __forceinline__ void plan_lcp(const PlanArgs &a, PlanSmem &sm, cooperative_groups::cluster_group &cluster, int e0,
                                         int e1) {
    constexpr int Q = 4;  // columns per lane and chunk
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int s0 = e0 + warp * EACH; s0 < e1; s0 += kWarps * EACH) {
        int n[EACH], far = 0;
        const int32_t *r0[EACH], *r1[EACH];
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int s = s0 + i, ld = s < e1 ? sm.leader[s] : -1;
            n[i] = ld >= 0 ? min(sm.full[s], sm.full[ld]) : 0;
            far = max(far, n[i]);
            r0[i] = a.table + (size_t)(ld >= 0 ? s : 0) * a.stride;
            r1[i] = a.table + (size_t)(ld >= 0 ? ld : 0) * a.stride;
        }
        for (int c0 = 0; c0 < far; c0 += 32 * Q) {
            int x[EACH][Q], y[EACH][Q];
#pragma unroll
            for (int i = 0; i < EACH; ++i)
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    const int c = max(min(c0 + 32 * q + lane, n[i] - 1), 0);
                    x[i][q] = r0[i][c];
                    y[i][q] = r1[i][c];
                }
            far = 0;
#pragma unroll
            for (int i = 0; i < EACH; ++i) {
                bool bad[Q], any = false;
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    bad[q] = x[i][q] != y[i][q] || (unsigned)x[i][q] >= (unsigned)a.n_total;
                    any |= bad[q];
                }
                if (c0 < n[i] && __any_sync(0xFFFFFFFFu, any)) {
#pragma unroll
                    for (int q = 0; q < Q; ++q) {
                        const unsigned m = __ballot_sync(0xFFFFFFFFu, bad[q]);
                        if (m) n[i] = min(n[i], c0 + 32 * q + __ffs(m) - 1);
                    }
                }
                if (n[i] > c0 + 32 * Q) far = max(far, n[i]);  // (a row that has differed reads no further)
            }
        }
        if (lane < kPlanCluster) {
#pragma unroll
            for (int i = 0; i < EACH; ++i)
                if (s0 + i < e1) *cluster.map_shared_rank(&sm.lcp[s0 + i], lane) = n[i];
        }
    }
}

// For each of the sequences [e0, e1) with a leader (and, MEMBERS, in a group), how many
// entries e of its class's part of seg count(e, s) holds for: done(s, leader, number).
// LANES lanes per sequence: a whole warp while a warp has one sequence, else 8, so that
// a warp's sequences are counted at the same time (2048 entries: 28.6 us in all, 31.2
// with 32).
template <int LANES, bool MEMBERS, typename Count, typename Done>
__device__ __forceinline__ void plan_per_class(const PlanSmem &sm, int e0, int e1, Count &&count, Done &&done) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int base = e0 + warp * (32 / LANES); base < e1; base += kPlanThreads / LANES) {
        const int s = base + lane / LANES;
        const int ld = s < e1 && (!MEMBERS || sm.member[s]) ? sm.leader[s] : -1;
        int n = 0;
        if (ld >= 0) {
            const int end = sm.cls_at[ld];
#pragma unroll 4
            for (int j = end - sm.cls_n[ld] + lane % LANES; j < end; j += LANES) n += count(sm.seg[j], s) ? 1 : 0;
        }
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
        if (s < e1 && lane % LANES == 0) done(s, ld, n);
    }
}

__global__ void __cluster_dims__(kPlanCluster, 1, 1) __launch_bounds__(kPlanThreads, 1)
    prefix_plan_kernel(const PlanArgs a) {
    extern __shared__ __align__(16) unsigned char plan_smem_raw[];
    PlanSmem &sm = *reinterpret_cast<PlanSmem *>(plan_smem_raw);
    auto cluster = cooperative_groups::this_cluster();
    const int tid = threadIdx.x;
    const int rank = (int)cluster.block_rank();
    const int B = a.B;
    const int e0 = (int)((long long)B * rank / kPlanCluster), e1 = (int)((long long)B * (rank + 1) / kPlanCluster);

    for (int i = tid; i < kPlanHash; i += kPlanThreads) {
        sm.key[i] = -1;
        sm.most[i] = 0;
        sm.lead[i] = kPlanMaxB;
    }
    __syncthreads();
    // leaders: every CTA hashes every sequence's first block
    for (int s = tid; s < B; s += kPlanThreads) {
        const int u = plan_full(a, s);
        sm.full[s] = u;
        const int first = u >= 1 ? a.table[(size_t)s * a.stride] : -1;
        int h = -1;
        if (first >= 0 && first < a.n_total) {
            h = (int)plan_hash(first);
            while (true) {  // at most B of twice as many slots are taken: a free one follows
                const int k = atomicCAS(&sm.key[h], -1, first);
                if (k == -1 || k == first) break;
                h = (h + 1) % kPlanHash;
            }
            atomicMax(&sm.most[h], u);
        }
        sm.leader[s] = h;  // hash slot for now
    }
    __syncthreads();
    for (int s = tid; s < B; s += kPlanThreads) {
        const int h = sm.leader[s];
        if (h >= 0 && sm.full[s] == sm.most[h]) atomicMin(&sm.lead[h], s);
    }
    __syncthreads();
    for (int s = tid; s < B; s += kPlanThreads) {
        const int h = sm.leader[s];
        sm.leader[s] = h < 0 ? -1 : sm.lead[h];
        sm.lcp[s] = 0;
    }
    cluster.sync();  // every CTA's arrays are ready for the others' writes
    // lcp of this CTA's sequences, given to every CTA; every sequence a warp has
    // is compared at the same time (their loads overlap)
    const int per_warp = (e1 - e0 + kWarps - 1) / kWarps;
    if (per_warp <= 1) plan_lcp<1>(a, sm, cluster, e0, e1);
    else plan_lcp<4>(a, sm, cluster, e0, e1);
    for (int s = tid; s < B; s += kPlanThreads) sm.cls_n[s] = 0;  // (the hash is no longer needed)
    cluster.sync();
    // the classes one after another, so that a sequence is compared with its own
    for (int s = tid; s < B; s += kPlanThreads)
        if (sm.leader[s] >= 0) atomicAdd(&sm.cls_n[sm.leader[s]], 1);
    __syncthreads();
    for (int base = 0, at = 0; base < B; base += kPlanThreads) {
        const int s = base + tid;
        const int n = s < B ? sm.cls_n[s] : 0;
        const int p = at + plan_scan(n, sm);
        if (s < B) sm.cls_at[s] = p;
        at += sm.total;
        __syncthreads();
    }
    for (int s = tid; s < B; s += kPlanThreads) {
        const int ld = sm.leader[s];
        if (ld >= 0) sm.seg[atomicAdd(&sm.cls_at[ld], 1)] = ((unsigned)sm.lcp[s] << 12) | (unsigned)s;
    }
    __syncthreads();  // (cls_at is now the class's end)
    // members of the class with at least this lcp, given to the first CTA
    {
        auto at_least = [&](unsigned e, int s) { return e >= (unsigned)sm.lcp[s] << 12; };
        auto give = [&](int s, int, int n) { *cluster.map_shared_rank(&sm.aux[s], 0) = n; };
        if (per_warp <= 1) plan_per_class<32, false>(sm, e0, e1, at_least, give);
        else plan_per_class<8, false>(sm, e0, e1, at_least, give);
    }
    cluster.sync();
    if (rank == 0) {
        // per class the most blocks saved, then the longest lcp that saves them
        for (int s = tid; s < B; s += kPlanThreads) {
            sm.gain[s] = 0;
            sm.shared[s] = 0;
            sm.gid[s] = B;
            sm.size[s] = 0;
        }
        __syncthreads();
        for (int s = tid; s < B; s += kPlanThreads)
            if (sm.leader[s] >= 0) atomicMax(&sm.gain[sm.leader[s]], (unsigned)sm.lcp[s] * (unsigned)(sm.aux[s] - 1));
        __syncthreads();
        for (int s = tid; s < B; s += kPlanThreads) {
            const int ld = sm.leader[s];
            if (ld >= 0 && (unsigned)sm.lcp[s] * (unsigned)(sm.aux[s] - 1) == sm.gain[ld]) atomicMax(&sm.shared[ld], sm.lcp[s]);
        }
        __syncthreads();
        for (int s = tid; s < B; s += kPlanThreads) {
            const int ld = sm.leader[s];
            bool in = false;
            if (ld >= 0) {
                const int p = sm.shared[ld];
                const unsigned cnt = sm.gain[ld] / (unsigned)p + 1;  // p >= 1: the first blocks are equal
                in = sm.lcp[s] >= p && p >= a.min_blocks && cnt >= (unsigned)a.min_members;
                if (in) {
                    atomicMin(&sm.gid[ld], s);
                    atomicAdd(&sm.size[ld], 1);
                }
                a.prefix_lens[s] = in ? p * a.b : 0;
            } else {
                a.prefix_lens[s] = 0;
            }
            sm.member[s] = in ? 1 : 0;
        }
        __syncthreads();
        // group numbers by lowest member, starts by the sizes: both in one scan
        int groups = 0, members = 0;
        for (int base = 0; base < B; base += kPlanThreads) {
            const int s = base + tid;
            const int ld = s < B ? sm.leader[s] : -1;
            const bool head = s < B && sm.member[s] && sm.gid[ld] == s;
            const int at = plan_scan(head ? (1 << 16) + sm.size[ld] : 0, sm);  // (at most 4096 members)
            const int total = sm.total;
            if (head) {
                const int g = groups + (at >> 16);
                a.group_start[g] = members + (at & 0xFFFF);
                a.group_blocks[g] = sm.shared[ld];
                sm.aux[ld] = members + (at & 0xFFFF);  // the class's first place (the counts are no longer needed)
            }
            groups += total >> 16;
            members += total & 0xFFFF;
            __syncthreads();
        }
        if (tid == 0) *a.n_groups = groups;
        for (int i = groups + tid; i <= B; i += kPlanThreads) a.group_start[i] = members;
        for (int i = groups + tid; i < B; i += kPlanThreads) a.group_blocks[i] = 0;
        for (int i = members + tid; i < B; i += kPlanThreads) a.members[i] = -1;
        __syncthreads();
    }
    cluster.sync();  // the first CTA's member flags and places
    // rank of each member inside its group: same leader, lower index
    if (rank != 0) {
        const PlanSmem *first = cluster.map_shared_rank(&sm, 0);
        for (int s = tid * 4; s < B; s += kPlanThreads * 4) {
            const unsigned m = *reinterpret_cast<const unsigned *>(first->member + s);
            const int4 p = *reinterpret_cast<const int4 *>(first->aux + s);
            *reinterpret_cast<unsigned *>(sm.member + s) = m;
            *reinterpret_cast<int4 *>(sm.aux + s) = p;
        }
        __syncthreads();
    }
    {
        auto before = [&](unsigned e, int s) {
            const int o = (int)(e & (kPlanMaxB - 1));
            return o < s && sm.member[o];
        };
        auto put = [&](int s, int ld, int n) {
            if (ld >= 0) a.members[sm.aux[ld] + n] = s;
        };
        if (per_warp <= 1) plan_per_class<32, true>(sm, e0, e1, before, put);
        else plan_per_class<8, true>(sm, e0, e1, before, put);
    }
    cluster.sync();  // the first CTA's shared memory outlives the others' reads
}

}  // namespace
}  // namespace zp

using namespace zp;

extern "C" zp_status zp_prefix_plan(const zp_cache_desc *D, const int32_t *block_table, int32_t table_stride,
                                    const int32_t *seq_lens, int32_t B, int32_t min_blocks, int32_t min_members,
                                    const zp_prefix_groups *plan, void *stream) {
    zp_status rc = check_desc(D);
    if (rc != ZP_OK) return rc;
    if (B < 0 || table_stride < 1 || min_blocks < 1 || min_members < 2)
        return fail(ZP_ERR_INVALID_ARG, "prefix_plan: B=%d table_stride=%d min_blocks=%d min_members=%d", B, table_stride,
                    min_blocks, min_members);
    if (!plan || !plan->n_groups || !plan->group_start ||
        (B > 0 && (!block_table || !seq_lens || !plan->prefix_lens || !plan->members || !plan->group_blocks)))
        return fail(ZP_ERR_INVALID_ARG, "prefix_plan: NULL buffer");
    if (B > kPlanMaxB) return fail(ZP_ERR_SHAPE, "prefix_plan: B %d > %d", B, kPlanMaxB);
    // (blocks saved by a class, stride * (B - 1), fit 32 bits)
    if (table_stride >= 1 << 20 || (long long)table_stride * D->block_size > INT32_MAX)
        return fail(ZP_ERR_SHAPE, "prefix_plan: table rows of %d blocks", table_stride);
    const PlanArgs a = {block_table, table_stride, seq_lens, B, D->block_size, D->n_total_blocks, min_blocks, min_members,
                        plan->prefix_lens, plan->n_groups, plan->group_start, plan->members, plan->group_blocks};
    rc = set_max_dynamic_smem(reinterpret_cast<const void *>(prefix_plan_kernel), sizeof(PlanSmem),
                              "prefix_plan: shared-memory attribute");
    if (rc != ZP_OK) return rc;
    prefix_plan_kernel<<<kPlanCluster, kPlanThreads, sizeof(PlanSmem), static_cast<cudaStream_t>(stream)>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "prefix_plan: launch");
    return ok();
}
