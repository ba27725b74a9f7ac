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
// a warp per sequence compares table rows, lcp and counts are exchanged through
// distributed shared memory, and the first CTA numbers the groups.  Bound by
// latency (four cluster barriers and the gather of the first column); the rows
// are read only up to their first difference.
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
    unsigned *err;
};

// Shared memory of one CTA.
struct PlanSmem {
    int key[kPlanHash];                  // first block id, -1 = free
    unsigned long long lead[kPlanHash];  // (u << 32) | ~index of the leader; later (gain, lcp) of the class
    int leader[kPlanMaxB];               // leader of each sequence, -1 = no class
    int lcp[kPlanMaxB];
    int aux[kPlanMaxB];                  // members with at least this lcp, then the rank inside the group
    int gid[kPlanMaxB];                  // by leader: lowest member, then group number
    int size[kPlanMaxB];                 // by leader: members
    int full[kPlanMaxB];                 // blocks before the newest token's
    unsigned char member[kPlanMaxB];
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

__global__ void __cluster_dims__(kPlanCluster, 1, 1) __launch_bounds__(kPlanThreads, 1)
    prefix_plan_kernel(const PlanArgs a) {
    extern __shared__ __align__(16) unsigned char plan_smem_raw[];
    PlanSmem &sm = *reinterpret_cast<PlanSmem *>(plan_smem_raw);
    auto cluster = cooperative_groups::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cluster.block_rank();
    const int B = a.B;
    const int e0 = (int)((long long)B * rank / kPlanCluster), e1 = (int)((long long)B * (rank + 1) / kPlanCluster);

    for (int i = tid; i < kPlanHash; i += kPlanThreads) {
        sm.key[i] = -1;
        sm.lead[i] = 0;
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
            atomicMax(&sm.lead[h], ((unsigned long long)u << 32) | (unsigned)(~s));
        }
        sm.leader[s] = h;  // hash slot for now
    }
    __syncthreads();
    for (int s = tid; s < B; s += kPlanThreads) {
        const int h = sm.leader[s];
        sm.leader[s] = h < 0 ? -1 : (int)~(unsigned)(sm.lead[h] & 0xFFFFFFFFull);
        sm.lcp[s] = 0;
    }
    cluster.sync();  // every CTA's arrays are ready for the others' writes
    // lcp of this CTA's sequences, given to every CTA: a warp compares kEach rows
    // with their leaders' at a time, 64 entries each, all loads in flight
    constexpr int kWarps = kPlanThreads / 32, kEach = 4;
    for (int s0 = e0 + warp * kEach; s0 < e1; s0 += kWarps * kEach) {
        int lim[kEach], n[kEach], far = 0;
        const int32_t *r0[kEach], *r1[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int s = s0 + i, ld = s < e1 ? sm.leader[s] : -1;
            lim[i] = ld >= 0 ? min(sm.full[s], sm.full[ld]) : 0;
            n[i] = lim[i];
            far = max(far, lim[i]);
            r0[i] = a.table + (size_t)(ld >= 0 ? s : 0) * a.stride;
            r1[i] = a.table + (size_t)(ld >= 0 ? ld : 0) * a.stride;
        }
        for (int c0 = 0; c0 < far; c0 += 64) {
            int x[kEach][2], y[kEach][2];
#pragma unroll
            for (int i = 0; i < kEach; ++i)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int c = c0 + 32 * q + lane;
                    const bool in = c < n[i];  // (a row that has differed reads no further)
                    x[i][q] = in ? r0[i][c] : 0;
                    y[i][q] = in ? r1[i][c] : 0;
                }
            far = 0;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const unsigned bad =
                        __ballot_sync(0xFFFFFFFFu, !(x[i][q] == y[i][q] && x[i][q] >= 0 && x[i][q] < a.n_total));
                    if (bad) n[i] = min(n[i], c0 + 32 * q + __ffs(bad) - 1);
                }
                far = max(far, n[i]);
            }
        }
        if (lane < kPlanCluster) {
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                if (s0 + i < e1) *cluster.map_shared_rank(&sm.lcp[s0 + i], lane) = n[i];
        }
    }
    cluster.sync();
    // members of the class with at least this lcp, given to the first CTA
    constexpr int kMany = 8;  // sequences a warp counts for together
    for (int s0 = e0 + warp * kMany; s0 < e1; s0 += kWarps * kMany) {
        int ld[kMany], n[kMany], cnt[kMany];
#pragma unroll
        for (int i = 0; i < kMany; ++i) {
            ld[i] = s0 + i < e1 ? sm.leader[s0 + i] : -1;
            n[i] = s0 + i < e1 ? sm.lcp[s0 + i] : 0;
            if (ld[i] < 0) ld[i] = -2;  // equal to no leader
            cnt[i] = 0;
        }
        for (int j = lane; j < B; j += 32) {
            const int lj = sm.leader[j], nj = sm.lcp[j];
#pragma unroll
            for (int i = 0; i < kMany; ++i) cnt[i] += lj == ld[i] && nj >= n[i] ? 1 : 0;
        }
#pragma unroll
        for (int i = 0; i < kMany; ++i) {
            const int c = __reduce_add_sync(0xFFFFFFFFu, cnt[i]);
            if (lane == 0 && s0 + i < e1) *cluster.map_shared_rank(&sm.aux[s0 + i], 0) = c;
        }
    }
    cluster.sync();
    if (rank == 0) {
        // best (blocks saved, lcp) and its member count per class
        for (int s = tid; s < B; s += kPlanThreads) sm.lead[s] = 0;
        __syncthreads();
        for (int s = tid; s < B; s += kPlanThreads) {
            const int ld = sm.leader[s];
            if (ld < 0) continue;
            const unsigned long long gain = (unsigned long long)sm.lcp[s] * (unsigned)(sm.aux[s] - 1);
            // gain < 2^31 * 2^12, lcp < 2^31 but at most the row length: 21 bits are left for it
            atomicMax(&sm.lead[ld], (gain << 21) | (unsigned)min(sm.lcp[s], (1 << 21) - 1));
            sm.gid[ld] = B;
            sm.size[ld] = 0;
        }
        __syncthreads();
        for (int s = tid; s < B; s += kPlanThreads) {
            const int ld = sm.leader[s];
            bool in = false;
            if (ld >= 0) {
                const int p = (int)(sm.lead[ld] & ((1u << 21) - 1));
                const unsigned long long gain = sm.lead[ld] >> 21;
                const unsigned long long cnt = gain / (unsigned)p + 1;  // p >= 1: the first blocks are equal
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
        // group numbers by lowest member; starts by a scan of the sizes
        int groups = 0, members = 0;
        for (int base = 0; base < B; base += kPlanThreads) {
            const int s = base + tid;
            const int ld = s < B ? sm.leader[s] : -1;
            const bool head = s < B && sm.member[s] && sm.gid[ld] == s;
            const int g = groups + plan_scan(head ? 1 : 0, sm);
            groups += sm.total;
            __syncthreads();
            const int at = members + plan_scan(head ? sm.size[ld] : 0, sm);
            members += sm.total;
            __syncthreads();
            if (head) {
                a.group_start[g] = at;
                a.group_blocks[g] = (int)(sm.lead[ld] & ((1u << 21) - 1));
                sm.aux[ld] = at;  // the class's first place (the counts are no longer needed)
            }
        }
        if (tid == 0) *a.n_groups = groups;
        for (int i = groups + tid; i <= B; i += kPlanThreads) a.group_start[i] = members;
        for (int i = groups + tid; i < B; i += kPlanThreads) a.group_blocks[i] = 0;
        for (int i = members + tid; i < B; i += kPlanThreads) a.members[i] = -1;
        __syncthreads();
    }
    cluster.sync();  // the first CTA's member flags and places
    // rank of each member inside its group: same leader, lower index
    const PlanSmem *first = cluster.map_shared_rank(&sm, 0);
    if (rank != 0) {
        for (int s = tid; s < e1; s += kPlanThreads) sm.member[s] = first->member[s];
        __syncthreads();
    }
    for (int s0 = e0 + warp * kMany; s0 < e1; s0 += kWarps * kMany) {
        int ld[kMany], r[kMany];
#pragma unroll
        for (int i = 0; i < kMany; ++i) {
            ld[i] = s0 + i < e1 && sm.member[s0 + i] ? sm.leader[s0 + i] : -2;
            r[i] = 0;
        }
        const int end = min(e1, s0 + kMany);
        for (int j = lane; j < end; j += 32) {
            const int lj = sm.member[j] ? sm.leader[j] : -1;
#pragma unroll
            for (int i = 0; i < kMany; ++i) r[i] += lj == ld[i] && j < s0 + i ? 1 : 0;
        }
#pragma unroll
        for (int i = 0; i < kMany; ++i) {
            const int c = __reduce_add_sync(0xFFFFFFFFu, r[i]);
            if (lane == 0 && ld[i] >= 0) a.members[first->aux[ld[i]] + c] = s0 + i;
        }
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
    if (table_stride >= 1 << 21 || (long long)table_stride * D->block_size > INT32_MAX)
        return fail(ZP_ERR_SHAPE, "prefix_plan: table rows of %d blocks", table_stride);
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != ZP_OK) return rc;
    const PlanArgs a = {block_table, table_stride, seq_lens, B, D->block_size, D->n_total_blocks, min_blocks, min_members,
                        plan->prefix_lens, plan->n_groups, plan->group_start, plan->members, plan->group_blocks,
                        dev.error_word};
    rc = set_max_dynamic_smem(reinterpret_cast<const void *>(prefix_plan_kernel), sizeof(PlanSmem),
                              "prefix_plan: shared-memory attribute");
    if (rc != ZP_OK) return rc;
    prefix_plan_kernel<<<kPlanCluster, kPlanThreads, sizeof(PlanSmem), static_cast<cudaStream_t>(stream)>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "prefix_plan: launch");
    return ok();
}
