// prefix_tc.cu -- the shared prefix on the fifth-generation tensor cores (bf16
// caches): the dense product of a group's query rows with its prefix, and the
// window score of the prefix tokens.  See prefix_attn.cu for the formulas and
// the split of the work.
//
// prefix_part_tc_kernel: one persistent CTA per SM.  An item has up to 256 query
// rows, two streams of 128 (one softmax warpgroup each, a thread per row):
//   S_w = Q_w K^T   (tcgen05.mma, both operands in shared memory, 128 x 128)
//   P_w = 2^(x - m) rounded to bf16, written over S_w in tensor memory
//   O_w += P_w V    (A = P_w from tensor memory, B = V as it lies, d contiguous)
// so that the tensor cores work on one stream while the other's softmax runs.
// An item with at most 128 rows gives both streams the same rows and every
// other tile of prefix tokens each; its pieces are joined like any others.
// Tensor memory: S_0, S_1 (128 columns each), O_0, O_1 (d columns each).  The
// running maximum m of a row is raised, and O_w rescaled, only when a tile
// exceeds it by more than 2^8 (the result does not depend on m, and P stays
// below 2^8); S_w of the next tile is complete only after O_w's last product,
// so the rescaling needs no wait of its own.
// K and V tiles of 128 tokens arrive by TMA with the 128-byte swizzle through a
// ring of stages, one copy per 16 token rows (a part of one block): the box is
// {64 elements, 8 tokens, d/64 halves, one head, 2 groups of 8 tokens}, so that
// in shared memory the halves of 8 tokens are 1024 bytes apart and the groups
// d/64 * 1024, a uniform stride for either operand.
//
// Bound by the chain of products and softmax: a tile's products take 2824 cycles
// (128 x 128 x 128 with both operands in shared memory 823, with A in tensor memory
// 589, twice each), a tile of 256 rows 3150 to 3600.  64 sequences behind 32k tokens
// (2048 query rows, 34 GFLOP, 134 MB of keys and values, 13.5 tiles per CTA): 35 us, of
// which 5 until the first logits, 25 the tiles (1.4 PFLOP/s, 5.3 TB/s), 4.6 the 20 MB
// of records.  Raising the maximum at every tile costs 1 us there, the test for a maximum
// so far from zero that its rounding would count 0.2 us.
#include <math.h>

#include "prefix_common.cuh"
#include "prefix_layout.h"
#include "prefix_tc.h"
#include "tc05.cuh"

namespace zp {
namespace {

constexpr int kPtTile = 128;                // prefix tokens per tile
constexpr int kPtThreads = 32 * (2 + 8);    // TMA, MMA, two warpgroups
constexpr int kPsEpi = 16;                  // epilogue warps of the score kernel
constexpr int kPsThreads = 32 * (2 + kPsEpi);
constexpr float kPtRaise = 8.f;             // log2 units a tile may exceed the running maximum by
constexpr float kPtFar = 67108864.f;        // 2^26: beyond, a maximum's rounding (half a step) passes 4 log2 units

// tcgen05.mma with A in tensor memory (bf16 pairs, one row per lane).
__device__ __forceinline__ void tc_mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Shared-memory descriptor of a K or V tile as the copies leave it: groups of 8
// tokens `group` bytes apart (stride offset).  K is contiguous along the product's
// K dimension; V along its N dimension, whose next 64 dims are 1024 bytes further
// (leading offset; not used by K).
__device__ __forceinline__ uint64_t sdesc_kv_sw128(uint32_t saddr, uint32_t group) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(1024u >> 4) << 16;
    d |= (uint64_t)(group >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// Stores to the warp's 32 TMEM lanes, waited for in the same statement.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};\n\t"
        "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

template <int D>
struct PtCfg {
    static constexpr int KH = D / 64;
    static constexpr int KS = D / 16;
    static constexpr int HALF = kPtTile * 128;        // bytes of 128 rows x 64 elements
    static constexpr int TILE = KH * HALF;            // a Q, K or V tile
    static constexpr int GROUP = KH * 1024;           // 8 tokens of a K or V tile
    static constexpr int STAGES = D == 128 ? 4 : 8;   // K and V tiles in flight
    static constexpr int Q_OFF = 0;                   // two query tiles
    static constexpr int ST_OFF = 2 * TILE;
    static constexpr int BAR_OFF = ST_OFF + STAGES * TILE;
    static constexpr int PRE_OFF = BAR_OFF + 512;
    static constexpr int smem(int B) { return PRE_OFF + (B + 1) * 4 + 1024; }
    static constexpr uint32_t TMEM_COLS = 512;
    static constexpr uint32_t S_COL = 0, O_COL = 256;
    static constexpr uint32_t IDESC_QK = idesc_bf16_f32(128, 128);
    static constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, D) | (1u << 16);  // B contiguous along N
};

// One CTA's share of an item.
struct PtSeg : PfxSeg {
    int rows;    // query rows of the item (<= 256)
    bool split;  // at most 128 rows: the streams take alternate tiles
};

__device__ __forceinline__ PtSeg pt_segment(const PfxArgs &a, const int *pre, int ng, int w, int w1) {
    PtSeg s;
    static_cast<PfxSeg &>(s) = pfx_segment(a, pre, ng, w, w1);
    s.rows = min(kPtRows, (s.g.n << a.G_log) - s.item * kPtRows);
    s.split = s.rows <= kPtRows / 2;
    return s;
}

// Tiles of stream w in a segment.
__device__ __forceinline__ int pt_tiles(const PtSeg &s, int w) {
    const int n = s.t_e - s.t_b;
    return s.split ? (n - w + 1) / 2 : n;
}

// First group of 8 rows ((block * b + slot) / 8) of the 16 tokens from `tok`; one
// outside the tensor (zeros are read) beyond the prefix and for a bad block.
__device__ __forceinline__ int pt_rows16(const PfxArgs &a, const PfxGroup &g, const int32_t *row, int tok) {
    if (tok >= g.tokens) return -2;
    const long long s = pfx_slot(a, row, tok);
    return s < 0 ? -2 : (int)(s / 8);
}

// Address of row r of the item's queries, nullptr beyond the last row.
template <int D>
__device__ __forceinline__ const uint4 *pt_query(const PfxArgs &a, const PtSeg &s, int head, int r, int *entry) {
    const int rr = s.item * kPtRows + r;
    *entry = r < s.rows ? pfx_member(a, s.g.m0 + (rr >> a.G_log)) : -1;
    if (*entry < 0) return nullptr;
    return reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) +
                                           ((size_t)*entry * a.h_q + (head << a.G_log) + (rr & (a.G - 1))) * D);
}

// The warp's 32 query rows (lane i holds the address of row row0 + i of the
// tile) into a swizzled tile of 64-element halves `half` bytes apart, a whole
// row per D/8 lanes; zeros for rows without an address.
template <int D>
__device__ __forceinline__ void pt_load_q(const uint4 *src, int row0, unsigned char *tile, int half) {
    constexpr int PER = D / 8;  // 16-byte chunks of a row
    const int lane = threadIdx.x & 31;
    uint4 v[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const uint4 *p = reinterpret_cast<const uint4 *>(
            __shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(src), i * (32 / PER) + lane / PER));
        v[i] = p ? __ldg(p + lane % PER) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int r = row0 + i * (32 / PER) + lane / PER, c = lane % PER;
        *reinterpret_cast<uint4 *>(tile + pt_chunk(r, c, half)) = v[i];
    }
}

template <int D>
__global__ void __launch_bounds__(kPtThreads, 1)
    prefix_part_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                          const PfxArgs a) {
    using C = PtCfg<D>;
    extern __shared__ unsigned char pt_raw[];
    unsigned char *smem =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(pt_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::BAR_OFF);
    uint64_t *empty = full + C::STAGES;
    uint64_t *q_full = empty + C::STAGES;  // [2] query tile written
    uint64_t *s_full = q_full + 2;         // [2] logits complete
    uint64_t *p_full = s_full + 2;         // [2][2] probabilities of the tile's first and last 64 tokens written
    uint64_t *o_full = p_full + 4;         // [2] last product of the segment complete
    uint64_t *drain = o_full + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *pre = reinterpret_cast<int *>(smem + C::PRE_OFF);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 4);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[2 * i], 4);
            mbar_init(&p_full[2 * i + 1], 4);
            mbar_init(&o_full[i], 1);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    const int ng = pfx_groups(a);
    const int W = pfx_scan(a, ng, pre);  // (ends with a barrier)
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (blockIdx.x == 0) pfx_publish(a, ng, pre);
    const int head = blockIdx.x % a.h_kv, set = blockIdx.x / a.h_kv;
    const int w0 = pfx_start(set, W, a.parts), w1 = pfx_start(set + 1, W, a.parts);

    if (warp < 2) pdl_trigger();
    if (warp == 0) {
        // ---------------- producer: K and V tiles in order
        uint32_t fill = 0;
        const int q = lane;  // lanes 0..7: 16 tokens each
        bool ok_all = true;
        if (lane == 0) {
            prefetch_tensormap(&kmap);
            prefetch_tensormap(&vmap);
        }
        for (int w = w0; w < w1 && ok_all;) {
            const PtSeg s = pt_segment(a, pre, ng, w, w1);
            w = s.w_e;
            if (s.t_b == s.t_e) continue;
            const int32_t *row = pfx_row(a, s.g);
            int z_next = lane < 8 ? pt_rows16(a, s.g, row, s.t_b * kPtTile + 16 * q) : 0;
            for (int t = s.t_b; t < s.t_e && ok_all; ++t) {
                const int z = z_next;
                if (t + 1 < s.t_e) z_next = lane < 8 ? pt_rows16(a, s.g, row, (t + 1) * kPtTile + 16 * q) : 0;
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const uint32_t st = fill % C::STAGES;
                    bool got = true;
                    if (lane == 0) {
                        got = mbar_wait_bounded(&empty[st], ((fill / C::STAGES) & 1) ^ 1, a.err, abort_flag, 0x601);
                        if (got) mbar_arrive_expect_tx(&full[st], C::TILE);
                    }
                    got = __shfl_sync(0xFFFFFFFFu, got ? 1 : 0, 0) != 0;
                    if (!got) {
                        ok_all = false;
                        break;
                    }
                    ++fill;
                    unsigned char *dst = smem + C::ST_OFF + st * C::TILE;
                    if (lane < 8) tma_load_5d(dst + q * 2 * C::GROUP, kv ? &vmap : &kmap, 0, 0, 0, head, z, &full[st]);
                    __syncwarp();
                }
            }
        }
        if (lane == 0 && *abort_flag) {  // copies in flight land before the CTA ends
            volatile int never = 0;
            for (uint32_t f = fill > C::STAGES ? fill - C::STAGES : 0; f < fill; ++f)
                mbar_wait_bounded(&full[f % C::STAGES], (f / C::STAGES) & 1, a.err, &never, 0x602);
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer (one thread)
        if (elect_one()) {
            uint32_t base = 0, n_p[2] = {0, 0}, n_q[2] = {0, 0};
            const uint32_t q_addr = smem_u32(smem + C::Q_OFF), st_addr = smem_u32(smem + C::ST_OFF);
            bool ok_all = true;
            for (int w = w0; w < w1 && ok_all;) {
                const PtSeg s = pt_segment(a, pre, ng, w, w1);
                w = s.w_e;
                if (s.t_b == s.t_e) continue;
                const int n_t[2] = {pt_tiles(s, 0), pt_tiles(s, 1)};
                // logits of stream x, its tile j
                auto qk = [&](int x, int j) -> bool {
                    const uint32_t f = base + 2 * (s.split ? 2 * j + x : j);
                    const uint32_t st = f % C::STAGES;
                    if (!mbar_wait_bounded(&full[st], (f / C::STAGES) & 1, a.err, abort_flag, 0x603)) return false;
                    tc_fence_after();
#pragma unroll
                    for (int ks = 0; ks < C::KS; ++ks) {
                        tc_mma_bf16(tmem + C::S_COL + x * 128,
                                    sdesc_k_sw128(q_addr + x * C::TILE + (ks >> 2) * C::HALF + (ks & 3) * 32),
                                    sdesc_kv_sw128(st_addr + st * C::TILE + (ks >> 2) * 1024 + (ks & 3) * 32, C::GROUP),
                                    C::IDESC_QK, ks > 0 ? 1u : 0u);
                    }
                    if (s.split || x == 1) tc_commit(&empty[st]);
                    tc_commit(&s_full[x]);
                    return true;
                };
                // the product of stream x's tile j with V, 64 tokens at a time as their
                // probabilities are written
                auto pv = [&](int x, int j) -> bool {
                    const uint32_t f = base + 2 * (s.split ? 2 * j + x : j) + 1;
                    const uint32_t st = f % C::STAGES;
                    if (!mbar_wait_bounded(&full[st], (f / C::STAGES) & 1, a.err, abort_flag, 0x604)) return false;
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        if (!mbar_wait_bounded(&p_full[2 * x + hf], n_p[x] & 1, a.err, abort_flag, 0x606)) return false;
                        tc_fence_after();
#pragma unroll
                        for (int ks = hf * 4; ks < hf * 4 + 4; ++ks)
                            tc_mma_bf16_ta(tmem + C::O_COL + x * D, tmem + C::S_COL + x * 128 + ks * 8,
                                           sdesc_kv_sw128(st_addr + st * C::TILE + ks * 2 * C::GROUP, C::GROUP), C::IDESC_PV,
                                           j > 0 || ks > 0 ? 1u : 0u);
                    }
                    ++n_p[x];
                    if (s.split || x == 1) tc_commit(&empty[st]);
                    return true;
                };
                for (int x = 0; x < 2 && ok_all; ++x) {
                    if (n_t[x] == 0) continue;
                    ok_all = mbar_wait_bounded(&q_full[x], n_q[x] & 1, a.err, abort_flag, 0x605);
                    ++n_q[x];
                    ok_all = ok_all && qk(x, 0);
                }
                for (int j = 0; j < n_t[0] && ok_all; ++j)  // n_t[0] >= n_t[1]
                    for (int x = 0; x < 2 && ok_all; ++x) {
                        if (j >= n_t[x]) continue;
                        ok_all = pv(x, j);
                        if (!ok_all) break;
                        if (j + 1 < n_t[x]) ok_all = qk(x, j + 1);
                        else tc_commit(&o_full[x]);
                    }
                base += 2 * (s.t_e - s.t_b);
            }
            // every product has been carried out before the CTA ends, also after a timeout
            volatile int never = 0;
            tc_commit(drain);
            mbar_wait_bounded(drain, 0, a.err, &never, 0x609);
        }
        __syncwarp();
    } else {
        // ---------------- softmax: warpgroup x = stream, thread = query row (TMEM lane)
        const int x = (warp - 2) >> 2;
        const int quarter = warp & 3;
        const int tr = quarter * 32 + lane;  // row of the tile
        const uint32_t lane_base = tmem + ((uint32_t)(32 * quarter) << 16);
        const uint32_t s_t = lane_base + C::S_COL + x * 128, o_t = lane_base + C::O_COL + x * D;
        uint32_t n_s = 0, n_o = 0;
        const float raise_by = kPtRaise / a.qscale;
        bool ok_all = true;
        for (int w = w0; w < w1 && ok_all;) {
            const PtSeg s = pt_segment(a, pre, ng, w, w1);
            w = s.w_e;
            if (s.t_b == s.t_e) continue;
            const int n_t = pt_tiles(s, x);
            const int r = s.split ? tr : x * 128 + tr;  // row of the item
            float vm = -INFINITY, l = 0.f;  // maximum of the products (logits / qscale), sum
            if (n_t > 0) {
                int entry;
                pt_load_q<D>(pt_query<D>(a, s, head, r, &entry), quarter * 32, smem + C::Q_OFF + x * C::TILE, C::HALF);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_full[x]);
            }
            for (int j = 0; j < n_t; ++j) {
                if (!mbar_wait_bounded(&s_full[x], n_s & 1, a.err, abort_flag, 0x607)) {
                    ok_all = false;
                    break;
                }
                ++n_s;
                tc_fence_after();
                const int t = s.t_b + (s.split ? 2 * j + x : j);
                const int valid = min(kPtTile, s.g.tokens - t * kPtTile);  // a multiple of 16
                uint32_t v0[64], v1[64];
                tmem_ld64(s_t, v0);
                tmem_ld64(s_t + 64, v1);
                if (valid < kPtTile) {
#pragma unroll
                    for (int c = 0; c < 64; ++c) {
                        if (c >= valid) v0[c] = 0xFF800000u;  // -inf
                        if (c + 64 >= valid) v1[c] = 0xFF800000u;
                    }
                }
                float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < 64; c += 2) {
                    mx4[c & 2] = fmaxf(mx4[c & 2], fmaxf(__uint_as_float(v0[c]), __uint_as_float(v0[c + 1])));
                    mx4[(c & 2) + 1] = fmaxf(mx4[(c & 2) + 1], fmaxf(__uint_as_float(v1[c]), __uint_as_float(v1[c + 1])));
                }
                const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
                // raise the maximum (and rescale what is summed) only beyond 2^8
                const bool raise = mx > vm + raise_by;  // true at the first tile with a logit above -inf
                if (__any_sync(0xFFFFFFFFu, raise)) {
                    const float al = raise ? (j == 0 ? 0.f : ex2_approx((vm - mx) * a.qscale)) : 1.f;
                    if (raise) vm = mx;
                    l *= al;
                    if (j > 0) {
#pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 32) {
                            uint32_t o[32];
                            tmem_ld32(o_t + c0, o);
#pragma unroll
                            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * al);
                            tmem_st32(o_t + c0, o);
                        }
                    }
                }
                // x - m in one rounding, m = vm qscale rounded.  No logit above -inf yet: every
                // probability is 2^(-inf), not 2^(-inf + inf).  Far from zero the rounding of m
                // alone would scale every probability: there the maximum is taken off first.
                float neg = vm == -INFINITY ? 0.f : -(vm * a.qscale);
                const bool far = fabsf(neg) > kPtFar;
                if (__any_sync(0xFFFFFFFFu, far)) {
                    const float off = far ? vm : 0.f;
#pragma unroll
                    for (int c = 0; c < 64; ++c) {
                        v0[c] = __float_as_uint(__uint_as_float(v0[c]) - off);
                        v1[c] = __float_as_uint(__uint_as_float(v1[c]) - off);
                    }
                    if (far) neg = 0.f;
                }
                const float2 sc = make_float2(a.qscale, a.qscale), nm = make_float2(neg, neg);
                float2 sum0 = make_float2(0.f, 0.f), sum1 = make_float2(0.f, 0.f);
                uint32_t p[32];
                auto half_tile = [&](const uint32_t(&v)[64], uint32_t col) {
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        float2 y = ffma2(make_float2(__uint_as_float(v[2 * c]), __uint_as_float(v[2 * c + 1])), sc, nm);
                        y.x = ex2_approx(y.x);
                        y.y = ex2_approx(y.y);
                        float2 &sum = c & 1 ? sum1 : sum0;
                        sum.x += y.x;
                        sum.y += y.y;
                        p[c] = f2_to_bf2(y.x, y.y);
                    }
                    tmem_st32(s_t + col, p);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[2 * x + col / 32]);
                };
                half_tile(v0, 0);
                half_tile(v1, 32);
                l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
            }
            if (!ok_all) break;
            pdl_trigger();  // (the decode does not read the records)
            // the piece's record: D/2 dims of the warp's 32 rows at a time through the bytes
            // of its own query rows (whose products are complete; the next item's queries
            // go to the same bytes), so that stores are whole 128-byte lines
            long long at = -1;
            if (r < s.rows)
                at = s.t_b == 0 ? pfx_main_row(a, s.g, head, s.item * kPtRows + r) + (s.split && x ? (long long)a.B * a.h_q : 0)
                                : a.extra0 + (long long)blockIdx.x * kPtRows + x * 128 + tr;
            if (n_t > 0) {
                if (!mbar_wait_bounded(&o_full[x], n_o & 1, a.err, abort_flag, 0x608)) break;
                ++n_o;
                tc_fence_after();
                unsigned char *buf = smem + C::Q_OFF + x * C::TILE;
                constexpr int COLS = pt_record_cols(D);
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += COLS) {
#pragma unroll
                    for (int c1 = 0; c1 < COLS; c1 += 32) {
                        uint32_t o[32];
                        tmem_ld32(o_t + c0 + c1, o);
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            *reinterpret_cast<uint4 *>(buf + pt_chunk(tr, c1 / 4 + c, C::HALF)) =
                                make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
                    }
                    __syncwarp();
                    constexpr int PER = COLS / 4;  // chunks per row
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        const int row = i * (32 / PER) + lane / PER, c = lane % PER;
                        const long long ra = __shfl_sync(0xFFFFFFFFu, at, row);
                        if (ra >= 0)
                            *reinterpret_cast<uint4 *>(a.rec_acc + ra * D + c0 + 4 * c) =
                                *reinterpret_cast<const uint4 *>(buf + pt_chunk(quarter * 32 + row, c, C::HALF));
                    }
                    __syncwarp();
                }
                tc_fence_before();
            }
            if (at >= 0) a.rec_ml[at] = make_float2(vm * a.qscale, l);
        }
    }

    __syncthreads();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, C::TMEM_COLS);
}

// ===========================================================================
// Window score of the prefix tokens: the 128 tokens of a tile are the M operand
// (a thread per token), the item's query rows the N operand, so the maximum over
// a kv head's q heads is taken in registers and consecutive lanes write
// consecutive tokens of a score row.  Accumulators of two tiles (256 columns
// each); per (token, sequence) one exponential of max_h (x_h - c_h),
// c = m + log2 l.  253 sequences behind 4k tokens, all on the first row of their window:
// 12 us from the statistics on for 33 MB of scores written, then 7 us for the 17 MB of
// logits of the private tokens; on a later row, 33 MB read as well, 3 us more.  No unit is
// full (over the kernel DRAM 14 % of its peak, L1 49 %, instructions in 48 % of the cycles):
// bound by the latency of the epilogue's chain from tensor memory to the stores.  Packed
// products and three-way maxima in it change nothing, with eight epilogue warps, not
// sixteen, the call takes 4 us more.
template <int D>
struct PsCfg {
    static constexpr int KH = D / 64;
    static constexpr int KS = D / 16;
    static constexpr int GROUP = KH * 1024;            // 8 tokens of a K tile
    static constexpr int TILE = kPtTile / 8 * GROUP;   // K tile
    static constexpr int B_HALF = kPtRows * 128;       // 256 query rows x 64 elements
    static constexpr int B_BYTES = KH * B_HALF;
    static constexpr int STAGES = 3;  // (leaves room for CTAs of the kernel before, so that this one starts beside it)
    static constexpr int ST_OFF = B_BYTES;
    static constexpr int BAR_OFF = ST_OFF + STAGES * TILE;
    static constexpr int C_OFF = BAR_OFF + 256;        // c of every row
    static constexpr int M_OFF = C_OFF + kPtRows * 4;  // score row of every member: offset * 2 + first, -1 none
    static constexpr int PRE_OFF = M_OFF + kPtRows * 8;
    static constexpr int smem(int B) { return PRE_OFF + (B + 1) * 4 + 1024; }
};

template <int D, int G>
__global__ void __launch_bounds__(kPsThreads, 1)
    prefix_score_tc_kernel(const __grid_constant__ CUtensorMap kmap, const PfxArgs a) {
    using C = PsCfg<D>;
    extern __shared__ unsigned char pt_raw[];
    unsigned char *smem =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(pt_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::BAR_OFF);
    uint64_t *empty = full + C::STAGES;
    uint64_t *q_full = empty + C::STAGES;  // the item's rows written (every epilogue warp)
    uint64_t *c_full = q_full + 1;         // its statistics and score rows too
    uint64_t *q_done = c_full + 1;         // the item finished by every epilogue warp
    uint64_t *acc_full = q_done + 1;       // [2]
    uint64_t *acc_empty = acc_full + 2;  // [2]
    uint64_t *drain = acc_empty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    float *cs = reinterpret_cast<float *>(smem + C::C_OFF);
    long long *ms = reinterpret_cast<long long *>(smem + C::M_OFF);
    int *pre = reinterpret_cast<int *>(smem + C::PRE_OFF);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(q_full, 8);  // (the first eight epilogue warps, a row per thread)
        mbar_init(c_full, 8);
        mbar_init(q_done, kPsEpi);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], kPsEpi);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    const int ng = pfx_groups(a);
    const int W = pfx_scan(a, ng, pre);
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int head = blockIdx.x % a.h_kv, set = blockIdx.x / a.h_kv;
    const int w0 = pfx_start(set, W, a.parts), w1 = pfx_start(set + 1, W, a.parts);

    if (warp == 0) {
        uint32_t fill = 0;
        const int q = lane;
        bool ok_all = true;
        if (lane == 0) prefetch_tensormap(&kmap);
        for (int w = w0; w < w1 && ok_all;) {
            const PtSeg s = pt_segment(a, pre, ng, w, w1);
            w = s.w_e;
            if (s.t_b == s.t_e) continue;
            const int32_t *row = pfx_row(a, s.g);
            for (int t = s.t_b; t < s.t_e; ++t, ++fill) {
                const int z = lane < 8 ? pt_rows16(a, s.g, row, t * kPtTile + 16 * q) : 0;
                const uint32_t st = fill % C::STAGES;
                bool got = true;
                if (lane == 0) {
                    got = mbar_wait_bounded(&empty[st], ((fill / C::STAGES) & 1) ^ 1, a.err, abort_flag, 0x611);
                    if (got) mbar_arrive_expect_tx(&full[st], C::TILE);
                }
                got = __shfl_sync(0xFFFFFFFFu, got ? 1 : 0, 0) != 0;
                if (!got) {
                    ok_all = false;
                    break;
                }
                if (lane < 8)
                    tma_load_5d(smem + C::ST_OFF + st * C::TILE + q * 2 * C::GROUP, &kmap, 0, 0, 0, head, z, &full[st]);
                __syncwarp();
            }
        }
        if (lane == 0 && *abort_flag) {
            volatile int never = 0;
            for (uint32_t f = fill > C::STAGES ? fill - C::STAGES : 0; f < fill; ++f)
                mbar_wait_bounded(&full[f % C::STAGES], (f / C::STAGES) & 1, a.err, &never, 0x612);
        }
    } else if (warp == 1) {
        if (elect_one()) {
            uint32_t fill = 0, n_q = 0;
            const uint32_t b_addr = smem_u32(smem), st_addr = smem_u32(smem + C::ST_OFF);
            bool ok_all = true;
            for (int w = w0; w < w1 && ok_all;) {
                const PtSeg s = pt_segment(a, pre, ng, w, w1);
                w = s.w_e;
                if (s.t_b == s.t_e) continue;
                const uint32_t idesc = idesc_bf16_f32(128, (s.rows + 15) / 16 * 16);
                ok_all = mbar_wait_bounded(q_full, n_q & 1, a.err, abort_flag, 0x613);
                ++n_q;
                for (int t = s.t_b; t < s.t_e && ok_all; ++t, ++fill) {
                    const uint32_t st = fill % C::STAGES, ab = fill & 1;
                    ok_all = mbar_wait_bounded(&full[st], (fill / C::STAGES) & 1, a.err, abort_flag, 0x614) &&
                             mbar_wait_bounded(&acc_empty[ab], ((fill >> 1) & 1) ^ 1, a.err, abort_flag, 0x615);
                    if (!ok_all) break;
                    tc_fence_after();
#pragma unroll
                    for (int ks = 0; ks < C::KS; ++ks)
                        tc_mma_bf16(tmem + ab * 256,
                                    sdesc_kv_sw128(st_addr + st * C::TILE + (ks >> 2) * 1024 + (ks & 3) * 32, C::GROUP),
                                    sdesc_k_sw128(b_addr + (ks >> 2) * C::B_HALF + (ks & 3) * 32), idesc, ks > 0 ? 1u : 0u);
                    tc_commit(&empty[st]);
                    tc_commit(&acc_full[ab]);
                }
            }
            volatile int never = 0;
            tc_commit(drain);
            mbar_wait_bounded(drain, 0, a.err, &never, 0x617);
        }
        __syncwarp();
    } else {
        const int et = threadIdx.x - 64;  // below 256: query row while loading
        const int quarter = warp & 3, col0 = ((warp - 2) >> 2) * (kPtRows * 4 / kPsEpi);  // lanes, 64 columns
        const float inv_w = 1.f / (float)a.window;
        uint32_t tile = 0, item = 0;
        bool ok_all = true, waited = false;
        // (every wait is bounded, so a warp that stops cannot leave another waiting for ever)
        for (int w = w0; w < w1 && ok_all;) {
            const PtSeg s = pt_segment(a, pre, ng, w, w1);
            w = s.w_e;
            if (s.t_b == s.t_e) continue;
            // the item's rows: once every warp has finished the last item (whose
            // products are then complete)
            if (!mbar_wait_bounded(q_done, (item & 1) ^ 1, a.err, abort_flag, 0x618)) break;
            int e = -1, row = -1;
            bool first = false;
            if (et < kPtRows) {
                pt_load_q<D>(pt_query<D>(a, s, head, et, &e), et & ~31, smem, C::B_HALF);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full);
                row = e >= 0 ? pfx_score_row(a, e, &first) : -1;
                // the scores that are added to, towards L2 while the records are joined
                if (et % G == 0 && row >= 0 && !first) {
                    const float *at = a.score + ((size_t)row * a.h_kv + head) * a.score_stride;
                    for (int tok = s.t_b * kPtTile; tok < min(s.t_e * kPtTile, s.g.tokens); tok += 32) prefetch_l2(at + tok);
                }
            }
            // only the statistics wait for the kernel that joins the records: the first
            // products run before it ends
            if (!waited) pdl_wait();
            waited = true;
            if (et < kPtRows) {
                float c = INFINITY;
                if (row >= 0) c = __ldcg(a.stats + (size_t)e * a.h_q + head * G + (s.item * kPtRows + et) % G);
                cs[et] = c;
                if (et % G == 0)
                    ms[et / G] = row >= 0 ? ((long long)row * a.h_kv + head) * a.score_stride * 2 + (first ? 1 : 0) : -1;
                __syncwarp();
                if (lane == 0) mbar_arrive(c_full);
            }
            if (!mbar_wait_bounded(c_full, item & 1, a.err, abort_flag, 0x619)) break;
            for (int t = s.t_b; t < s.t_e; ++t, ++tile) {
                const uint32_t ab = tile & 1;
                if (!mbar_wait_bounded(&acc_full[ab], (tile >> 1) & 1, a.err, abort_flag, 0x616)) {
                    ok_all = false;
                    break;
                }
                tc_fence_after();
                const int tok = t * kPtTile + 32 * quarter + lane;
                const uint32_t acc = tmem + ((uint32_t)(32 * quarter) << 16) + ab * 256 + col0;
                const bool live = tok < s.g.tokens;
                float *col = a.score + tok;
#pragma unroll 1
                for (int c0 = 0; c0 < kPtRows * 4 / kPsEpi; c0 += 16) {
                    if (col0 + c0 >= s.rows) break;
                    uint32_t v[16];
                    tmem_ld16(acc + c0, v);
                    constexpr int N = 16 / G;
                    float c[16];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<float4 *>(c + 4 * j) = reinterpret_cast<const float4 *>(cs + col0 + c0)[j];
                    long long mr[N];
#pragma unroll
                    for (int i = 0; i < N; ++i) mr[i] = ms[(col0 + c0) / G + i];
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        float x[G];
#pragma unroll
                        for (int j = 0; j < G; ++j)  // (x rounded as in the statistics: a maximum's x - c is never above -log2 l)
                            x[j] = __fmul_rn(__uint_as_float(v[i * G + j]), a.qscale) - c[i * G + j];
#pragma unroll
                        for (int o = 1; o < G; o <<= 1)
#pragma unroll
                            for (int j = 0; j < G; j += 2 * o) x[j] = fmaxf(x[j], x[j + o]);
                        pfx_put_score(col + (mr[i] >> 1), ex2_approx(x[0]) * inv_w, live && mr[i] >= 0, mr[i] & 1);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_empty[ab]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(q_done);
            ++item;
        }
        if (!waited) pdl_wait();
        if (ok_all) pfx_own_scores<G, 32 * kPsEpi>(a, et);
    }
    __syncthreads();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

zp_status pt_map(CUtensorMap *map, const void *base, const PfxArgs &a, int d) {
    const uint64_t row = (uint64_t)a.h_kv * d * 2;  // bytes of a token, every kv head
    const uint64_t dims[5] = {64, 8, (uint64_t)d / 64, (uint64_t)a.h_kv, (uint64_t)a.n_total * a.b / 8};
    const uint64_t strides[4] = {row, 128, (uint64_t)d * 2, 8 * row};
    const uint32_t box[5] = {64, 8, (uint32_t)d / 64, 1, 2};
    return encode_tmap_bf16(map, 5, base, dims, strides, box, "prefix_decode");
}

template <int D>
zp_status launch_part_tc(const PfxArgs &a, cudaStream_t st) {
    CUtensorMap km, vm;
    zp_status rc = pt_map(&km, a.k, a, D);
    if (rc != ZP_OK) return rc;
    rc = pt_map(&vm, a.v, a, D);
    if (rc != ZP_OK) return rc;
    const size_t smem = PtCfg<D>::smem(a.B);
    rc = set_max_dynamic_smem(reinterpret_cast<const void *>(prefix_part_tc_kernel<D>), smem,
                              "prefix_decode: shared-memory attribute");
    if (rc != ZP_OK) return rc;
    prefix_part_tc_kernel<D><<<a.parts * a.h_kv, kPtThreads, smem, st>>>(km, vm, a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "prefix_decode: prefix kernel launch");
    return ZP_OK;
}

template <int D, int G>
zp_status launch_score_tc(const PfxArgs &a, cudaStream_t st) {
    CUtensorMap km;
    zp_status rc = pt_map(&km, a.k, a, D);
    if (rc != ZP_OK) return rc;
    const size_t smem = PsCfg<D>::smem(a.B);
    rc = set_max_dynamic_smem(reinterpret_cast<const void *>(prefix_score_tc_kernel<D, G>), smem,
                              "prefix_decode: shared-memory attribute");
    if (rc != ZP_OK) return rc;
    const cudaError_t e = launch_dependent(prefix_score_tc_kernel<D, G>, dim3(a.parts * a.h_kv), dim3(kPsThreads), smem, st,
                                           km, a);
    if (e != cudaSuccess) return cuda_fail(e, "prefix_decode: score kernel launch");
    return ZP_OK;
}

}  // namespace

zp_status prefix_part_tc(const PfxArgs &a, int d, cudaStream_t st) {
    return d == 64 ? launch_part_tc<64>(a, st) : launch_part_tc<128>(a, st);
}

zp_status prefix_score_tc(const PfxArgs &a, int d, cudaStream_t st) {
    const int G = a.G;
    if (d == 64) {
        if (G == 1) return launch_score_tc<64, 1>(a, st);
        if (G == 2) return launch_score_tc<64, 2>(a, st);
        if (G == 4) return launch_score_tc<64, 4>(a, st);
        return launch_score_tc<64, 8>(a, st);
    }
    if (G == 1) return launch_score_tc<128, 1>(a, st);
    if (G == 2) return launch_score_tc<128, 2>(a, st);
    if (G == 4) return launch_score_tc<128, 4>(a, st);
    return launch_score_tc<128, 8>(a, st);
}

}  // namespace zp
