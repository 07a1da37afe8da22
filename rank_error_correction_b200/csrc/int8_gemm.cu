// int8_gemm.cu -- W8A8 for larger T on the 5th-generation tensor cores:
// tcgen05.mma kind::i8 on CTA pairs, int32 accumulators in TMEM.
//
//   y[t][o] = s_t s_o sum_k c[t][k] q[o][k] + sum_j R[t][j] A[o][j]
//
// A cluster of two CTAs computes 256 rows of W x BN tokens: CTA p stages rows
// [128 p, +128) of the codes and half of the tokens' codes (128-byte rows, one
// swizzle atom, by TMA), the leader's MMA thread issues M = 256, N = BN, K = 32
// per step, and each CTA's TMEM receives the int32 sums of its 128 rows.  The
// correction is K = 64 slabs of fp16 (A_i and R by TMA, zero beyond r) into
// fp32 columns of their own beside the sums, because one accumulator cannot
// hold both; the epilogue joins them in fp32 and rounds once.  Both are double
// buffered, so a tile's drain overlaps the next tile's products.
// When the tiles alone would not occupy every pair, the k of each tile is
// split into parts: every part stores its sums, and the part that counts last
// on the tile's ticket adds them (integers: the order does not matter).
#include <cstring>

#include "internal.cuh"
#include "tc.cuh"

namespace glowq {

constexpr int kI8Rows = 128;             // W rows per CTA (TMEM lanes)
constexpr int kI8Block = 128;            // k per stage: one 128-byte swizzle atom of int8
constexpr int kI8WBytes = kI8Rows * kI8Block;
constexpr int kI8Threads = 256;          // producer, MMA, forwarder, (idle), 4 epilogue warps
constexpr int kI8Chunk = 32;             // tokens per epilogue step
constexpr int kI8EpiBytes = kI8Chunk * kI8Rows * 2;
constexpr int kI8SmemMax = 227 * 1024;

template <int BN>
struct I8Tile {
    static constexpr int kHalf = BN / 2;
    static constexpr int kXBytes = kHalf * kI8Block;
    static constexpr int kStageBytes = kI8WBytes + kXBytes;
    static constexpr int kStages = BN == 256 ? 6 : BN == 128 ? 8 : 9;
    static constexpr int kCols = 4 * BN <= 512 ? 4 * BN : 512;   // two int32 and two fp32 accumulators
    static constexpr int kSmem = kStages * kStageBytes + 2 * kI8EpiBytes + 2 * BN * 4 + 512 + 1024;
    static_assert(BN % 64 == 0 && 4 * BN <= 512, "two accumulators of each kind in TMEM");
    static_assert(kSmem <= kI8SmemMax, "shared memory per CTA");
};

struct I8GemmModule {
    const float* s;
    int O;
    int mtile_begin;
    int has_A;
};
struct I8GemmArgs {
    CUtensorMap tmX;                       // codes [T][d], box {128, BN/2}, SW128
    CUtensorMap tmR;                       // R [T][r] fp16, box {64, BN/2}, SW128
    CUtensorMap tmW[GLOWQ_MAX_MODULES];    // codes [O][d], box {128, 128}, SW128
    CUtensorMap tmA[GLOWQ_MAX_MODULES];    // A [O][r] fp16, box {64, 128}, SW128
    CUtensorMap tmY[GLOWQ_MAX_MODULES];    // Y [T][ldY] fp16 (O columns), box {128, 32}
    I8GemmModule mod[GLOWQ_MAX_MODULES];
    const float* xs;
    int m, d, T, r;
    int ntiles_n, nunits;
    int S, kbs;                            // parts per tile, k-blocks per part
    int4* slots;                           // [tile][2 CTAs][S sums (+ 1 correction)][BN / 4][128 rows]
    unsigned int* tickets;                 // [tile][2 CTAs], zero between calls
    unsigned int* status;
};

struct __align__(8) I8Barriers {
    uint64_t full[9];          // per CTA: its TMA bytes landed
    uint64_t ready[9];         // leader: both CTAs' bytes landed (one arrival from each)
    uint64_t empty[9];         // per CTA: the pair's MMAs that read the stage completed
    uint64_t acc_full[2];      // per CTA: accumulators complete
    uint64_t acc_empty[2];     // leader: both CTAs drained them (one arrival per epilogue warp)
    uint32_t tmem_base;
    uint32_t last_part;
};

// Instruction descriptor, kind::i8: signed int8 A and B, int32 accumulator, both K-major, shape M x N.
__host__ __device__ constexpr uint32_t i8_idesc(int M, int N) {
    return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

struct I8Unit {
    int mi, m0, n0, tile, part;
    int kb0, nkb, nslab;
};
template <int BN>
__device__ __forceinline__ I8Unit i8_unit(const I8GemmArgs& a, int u) {
    I8Unit c;
    c.tile = u / a.S;
    c.part = u - c.tile * a.S;
    const int mt = c.tile / a.ntiles_n, nt = c.tile - mt * a.ntiles_n;
    c.mi = 0;
    for (int i = 1; i < a.m; ++i)
        if (mt >= a.mod[i].mtile_begin) c.mi = i;
    c.m0 = (mt - a.mod[c.mi].mtile_begin) * 2 * kI8Rows;
    c.n0 = nt * BN;
    const int all = a.d / kI8Block;
    c.kb0 = c.part * a.kbs;
    c.nkb = min(a.kbs, all - c.kb0);
    c.nslab = (c.part == 0 && a.r > 0 && a.mod[c.mi].has_A) ? (a.r + 63) / 64 : 0;
    return c;
}

// Four MMAs of one stage (32 bytes of k each), the commits that free it in both
// CTAs, and a non-blocking probe of the next stage's barrier whose round trip
// the issue hides.
template <bool INT>
__device__ __forceinline__ uint32_t i8_stage_mma(uint32_t dacc, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                 uint32_t accumulate, uint32_t empty_local, uint32_t empty_peer,
                                                 uint32_t probe_bar, uint32_t probe_parity) {
    uint32_t ready;
#define GLOWQ_STAGE_MMA(KIND)                                                                             \
    asm volatile(                                                                                         \
        "{\n\t.reg .pred pr, pa, pt;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"                             \
        "mbarrier.test_wait.parity.shared::cta.b64 pr, [%6], %7;\n\t"                                     \
        "setp.ne.b32 pa, %3, 0;\n\t"                                                                      \
        "setp.eq.b32 pt, %3, %3;\n\t"                                                                     \
        "add.s64 a1, %8, 2;\n\tadd.s64 a2, %8, 4;\n\tadd.s64 a3, %8, 6;\n\t"                              \
        "add.s64 b1, %9, 2;\n\tadd.s64 b2, %9, 4;\n\tadd.s64 b3, %9, 6;\n\t"                              \
        "tcgen05.mma.cta_group::2.kind::" KIND " [%1], %8, %9, %2, pa;\n\t"                               \
        "tcgen05.mma.cta_group::2.kind::" KIND " [%1], a1, b1, %2, pt;\n\t"                               \
        "tcgen05.mma.cta_group::2.kind::" KIND " [%1], a2, b2, %2, pt;\n\t"                               \
        "tcgen05.mma.cta_group::2.kind::" KIND " [%1], a3, b3, %2, pt;\n\t"                               \
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t"                 \
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%5];\n\t"                 \
        "selp.u32 %0, 1, 0, pr;\n\t}"                                                                     \
        : "=r"(ready)                                                                                     \
        : "r"(dacc), "r"(idesc), "r"(accumulate), "r"(empty_local), "r"(empty_peer), "r"(probe_bar),      \
          "r"(probe_parity), "l"(adesc), "l"(bdesc)                                                       \
        : "memory")
    if constexpr (INT) {
        GLOWQ_STAGE_MMA("i8");
    } else {
        GLOWQ_STAGE_MMA("f16");
    }
#undef GLOWQ_STAGE_MMA
    return ready;
}

template <int BN>
__global__ void __launch_bounds__(kI8Threads, 1) int8_gemm_kernel(const __grid_constant__ I8GemmArgs a) {
    using TL = I8Tile<BN>;
    constexpr int kStages = TL::kStages;
    extern __shared__ __align__(1024) unsigned char raw[];
    unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    unsigned char* epi = sm + kStages * TL::kStageBytes;
    float* tok = reinterpret_cast<float*>(epi + 2 * kI8EpiBytes);          // token scales of the tile
    I8Barriers* bars = reinterpret_cast<I8Barriers*>(tok + 2 * BN);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t crank = cluster_ctarank();                              // 0 = leader (issues the MMAs)
    const int first = (int)cluster_id_x(), step = (int)cluster_count_x();
    const int row_off = (int)crank * kI8Rows, tok_off = (int)crank * TL::kHalf;

    if (threadIdx.x == 32) {
        prefetch_tmap(&a.tmX);
        if (a.r > 0) prefetch_tmap(&a.tmR);
        for (int i = 0; i < a.m; ++i) {
            prefetch_tmap(&a.tmW[i]);
            if (a.mod[i].has_A) prefetch_tmap(&a.tmA[i]);
            prefetch_tmap(&a.tmY[i]);
        }
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->ready[s], 2);
            mbar_init(&bars->empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&bars->acc_full[b], 1);
            mbar_init(&bars->acc_empty[b], 8);
        }
        fence_mbar_init();
    }
    cluster_sync_all();
    if (warp == 1) tmem_alloc_pair(&bars->tmem_base, TL::kCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    pdl_launch_dependents();

    if (warp == 0) {
        // ---------------- producer (both CTAs) ----------------
        // The codes of W are static: the first ring of them is fetched before
        // the kernels that quantise X and compute R are known to be complete.
        if (lane == 0) {
            bool ok = true;
            int g = 0, early = 0;
            for (int pass = 0; pass < 2; ++pass) {
                g = 0;
                for (int unit = first; unit < a.nunits; unit += step) {
                    const I8Unit c = i8_unit<BN>(a, unit);
                    for (int i = 0; i < c.nkb + c.nslab; ++i, ++g) {
                        if (pass == 0 && (g >= kStages || i >= c.nkb)) goto stop;   // (slab stages are not static)
                        const int s = g % kStages;
                        if (g >= kStages && ok) ok = mbar_wait(&bars->empty[s], ((g / kStages) - 1) & 1, a.status);
                        const uint32_t ws = smem_u32(sm + s * TL::kStageBytes), xs = ws + kI8WBytes;
                        if (i < c.nkb) {
                            if (pass == 0 || g >= early) {
                                mbar_arrive_expect_tx(&bars->full[s], TL::kStageBytes);
                                tma_load_2d(ws, &a.tmW[c.mi], &bars->full[s], (c.kb0 + i) * kI8Block, c.m0 + row_off);
                            }
                            if (pass == 0) early = g + 1;
                            else tma_load_2d(xs, &a.tmX, &bars->full[s], (c.kb0 + i) * kI8Block, c.n0 + tok_off);
                        } else {
                            const int j = i - c.nkb;
                            mbar_arrive_expect_tx(&bars->full[s], TL::kStageBytes);
                            tma_load_2d(ws, &a.tmA[c.mi], &bars->full[s], j * 64, c.m0 + row_off);
                            tma_load_2d(xs, &a.tmR, &bars->full[s], j * 64, c.n0 + tok_off);
                        }
                    }
                }
            stop:
                if (pass == 0) pdl_wait();
            }
            // the leader's commits for the last stages land here before this CTA may exit
            for (int p = (g > kStages ? g - kStages : 0); p < g && ok; ++p)
                ok = mbar_wait(&bars->empty[p % kStages], (p / kStages) & 1, a.status);
        }
    } else if (warp == 2) {
        // ---------------- forwarder (both CTAs): own bytes landed -> the leader's barrier ----------------
        if (lane == 0) {
            bool ok = true;
            int g = 0;
            pdl_wait();                                   // (bounded waits begin when the codes of X can come)
            for (int unit = first; unit < a.nunits; unit += step) {
                const I8Unit c = i8_unit<BN>(a, unit);
                for (int i = 0; i < c.nkb + c.nslab; ++i, ++g) {
                    const int s = g % kStages;
                    if (ok) ok = mbar_wait(&bars->full[s], (g / kStages) & 1, a.status);
                    mbar_arrive_remote(cluster_addr(&bars->ready[s], 0));
                }
            }
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer (leader CTA) ----------------
        if (crank == 0 && lane == 0) {
            constexpr uint64_t kStageDesc = (uint64_t)(TL::kStageBytes >> 4);
            const uint64_t wdesc = sw128_kmajor_desc(smem_u32(sm));
            const uint64_t xdesc = sw128_kmajor_desc(smem_u32(sm) + kI8WBytes);
            const uint32_t empty_l = smem_u32(&bars->empty[0]), empty_p = cluster_addr(&bars->empty[0], 1);
            const uint32_t ready0 = smem_u32(&bars->ready[0]);
            bool ok = true, next_ready = false;
            pdl_wait();
            int tl = 0, s = 0;
            uint32_t ph = 0;
            for (int unit = first; unit < a.nunits; unit += step, ++tl) {
                const I8Unit c = i8_unit<BN>(a, unit);
                const int buf = tl & 1;
                if (tl >= 2 && ok) ok = mbar_wait_cluster(&bars->acc_empty[buf], ((tl >> 1) - 1) & 1, a.status);
                tc_fence_after();
                const uint32_t iacc = tmem + (uint32_t)(buf * BN), facc = tmem + (uint32_t)((2 + buf) * BN);
                for (int i = 0; i < c.nkb + c.nslab; ++i) {
                    if (!next_ready && ok) ok = mbar_wait_cluster(&bars->ready[s], ph, a.status);
                    tc_fence_after();
                    const int sn = (s + 1 == kStages) ? 0 : s + 1;
                    const uint32_t phn = (s + 1 == kStages) ? (ph ^ 1u) : ph;
                    const uint64_t ad = wdesc + (uint64_t)s * kStageDesc, bd = xdesc + (uint64_t)s * kStageDesc;
                    const uint32_t el = empty_l + 8u * (uint32_t)s, ep = empty_p + 8u * (uint32_t)s;
                    const uint32_t pb = ready0 + 8u * (uint32_t)sn;
                    if (i < c.nkb)
                        next_ready = i8_stage_mma<true>(iacc, ad, bd, i8_idesc(2 * kI8Rows, BN), i > 0, el, ep, pb, phn) != 0;
                    else
                        next_ready = i8_stage_mma<false>(facc, ad, bd, f16_idesc(2 * kI8Rows, BN), i > c.nkb, el, ep, pb, phn) != 0;
                    s = sn;
                    ph = phn;
                }
                umma_commit_pair(smem_u32(&bars->acc_full[buf]));
                umma_commit_pair(cluster_addr(&bars->acc_full[buf], 1));
            }
            for (int t = (tl > 2 ? tl - 2 : 0); t < tl && ok; ++t)
                ok = mbar_wait_cluster(&bars->acc_empty[t & 1], (t >> 1) & 1, a.status);
        }
    } else if (warp >= 4) {
        // ---------------- epilogue (warps 4..7, both CTAs), one thread per row ----------------
        const int quarter = warp & 3, row = quarter * 32 + lane, et = threadIdx.x - 128;
        const bool leader = et == 0;
        bool ok = true;
        int tl = 0, chunk = 0;
        pdl_wait();                                       // the token scales are complete
        for (int unit = first; unit < a.nunits; unit += step, ++tl) {
            const I8Unit c = i8_unit<BN>(a, unit);
            const int buf = tl & 1;
            const int orow = c.m0 + row_off + row;
            const float so = orow < a.mod[c.mi].O ? __ldg(a.mod[c.mi].s + orow) : 0.f;
            float* ts = tok + buf * BN;                   // (the previous tile's readers passed this tile's first barrier)
            for (int i = et; i < BN; i += 128) ts[i] = c.n0 + i < a.T ? ldcg_f32(a.xs + c.n0 + i) : 0.f;
            if (ok) ok = mbar_wait(&bars->acc_full[buf], (tl >> 1) & 1, a.status);
            tc_fence_after();
            named_barrier_sync(1, 128);                   // token scales staged
            const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
            const uint32_t iacc = tmem + lanes + (uint32_t)(buf * BN), facc = tmem + lanes + (uint32_t)((2 + buf) * BN);
            const bool slab_tile = a.r > 0 && a.mod[c.mi].has_A;
            // y of one chunk from its sums and correction
            auto store_chunk = [&](const uint32_t (&v)[32], const float (&f)[32], int ch) {
                unsigned char* sb = epi + (chunk & 1) * kI8EpiBytes;
                ++chunk;
                if (leader) bulk_wait_read<1>();
                named_barrier_sync(1, 128);
                __half* col = reinterpret_cast<__half*>(sb) + row;
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    col[j * kI8Rows] = __float2half_rn(fmaf((float)(int)v[j] * ts[ch * kI8Chunk + j], so, f[j]));
                fence_proxy_async_smem();
                named_barrier_sync(1, 128);
                const int o0 = c.m0 + row_off, t0 = c.n0 + ch * kI8Chunk;
                if (leader) {
                    if (o0 < a.mod[c.mi].O && t0 < a.T) tma_store_2d(&a.tmY[c.mi], smem_u32(sb), o0, t0);
                    bulk_commit();
                }
            };
            if (a.S == 1) {
#pragma unroll 1
                for (int ch = 0; ch < BN / kI8Chunk; ++ch) {
                    uint32_t v[32];
                    float f[32];
                    tmem_ld32(iacc + ch * kI8Chunk, v);
                    if (slab_tile) {
                        uint32_t w[32];
                        tmem_ld32(facc + ch * kI8Chunk, w);
#pragma unroll
                        for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(w[j]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) f[j] = 0.f;
                    }
                    store_chunk(v, f, ch);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(cluster_addr(&bars->acc_empty[buf], 0));
                continue;
            }
            // a part of a split tile: its sums to its slot ([token / 4][row] of 16 bytes), part 0's correction behind them
            const int per = a.S + (a.r > 0 ? 1 : 0);
            int4* slots = a.slots + ((int64_t)c.tile * 2 + crank) * per * (BN / 4 * kI8Rows) + row;
            auto to_slot = [&](uint32_t acc, int p) {
#pragma unroll 1
                for (int ch = 0; ch < BN / kI8Chunk; ++ch) {
                    uint32_t v[32];
                    tmem_ld32(acc + ch * kI8Chunk, v);
                    int4* dst = slots + ((int64_t)p * (BN / 4) + ch * 8) * kI8Rows;
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        __stcg(dst + q * kI8Rows, make_int4((int)v[4 * q], (int)v[4 * q + 1], (int)v[4 * q + 2], (int)v[4 * q + 3]));
                }
            };
            to_slot(iacc, c.part);
            if (c.nslab > 0) to_slot(facc, a.S);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(cluster_addr(&bars->acc_empty[buf], 0));
            __threadfence();
            named_barrier_sync(1, 128);
            if (leader) {
                unsigned int* tk = a.tickets + c.tile * 2 + crank;
                unsigned int prev;
                asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(prev) : "l"(tk) : "memory");
                const uint32_t last = prev == (unsigned)(a.S - 1) ? 1u : 0u;
                if (last) atomicExch(tk, 0u);             // every part has counted: ready for the next call
                *reinterpret_cast<volatile uint32_t*>(&bars->last_part) = last;
            }
            named_barrier_sync(1, 128);
            if (*reinterpret_cast<volatile uint32_t*>(&bars->last_part) == 0u) continue;
            __threadfence();
#pragma unroll 1
            for (int ch = 0; ch < BN / kI8Chunk; ++ch) {
                uint32_t v[32];
                float f[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = 0u, f[j] = 0.f;
#pragma unroll 1
                for (int p = 0; p < a.S; ++p) {
                    const int4* src = slots + ((int64_t)p * (BN / 4) + ch * 8) * kI8Rows;
                    int4 x[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) x[q] = __ldcg(src + q * kI8Rows);
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        v[4 * q] += (uint32_t)x[q].x;
                        v[4 * q + 1] += (uint32_t)x[q].y;
                        v[4 * q + 2] += (uint32_t)x[q].z;
                        v[4 * q + 3] += (uint32_t)x[q].w;
                    }
                }
                if (slab_tile) {
                    const int4* src = slots + ((int64_t)a.S * (BN / 4) + ch * 8) * kI8Rows;
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const int4 x = __ldcg(src + q * kI8Rows);
                        f[4 * q] = __int_as_float(x.x);
                        f[4 * q + 1] = __int_as_float(x.y);
                        f[4 * q + 2] = __int_as_float(x.z);
                        f[4 * q + 3] = __int_as_float(x.w);
                    }
                }
                store_chunk(v, f, ch);
            }
        }
        if (leader) bulk_wait_all();
    }
    pdl_wait();                                           // every thread: this grid's end implies the preceding ones'
    tc_fence_before();
    __syncwarp();
    cluster_sync_all();                                   // no arrivals or MMA reads into either CTA remain
    if (warp == 1) tmem_dealloc_pair(tmem, TL::kCols);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// Token width and parts per tile: the busiest pair's time in tensor-core
// clocks, a k-block of a tile costing its MMAs (2 BN) but not less than its
// codes' way from memory, a unit a fixed drain, a split its partial sums.
I8GemmPlan plan_int8_gemm(int64_t T, int64_t d, int64_t mtiles, int r, int num_sms) {
    I8GemmPlan best = {};
    const int64_t pairs = num_sms / 2 > 0 ? num_sms / 2 : 1, nkb = d / kI8Block;
    double least = 0;
    for (int bn = 64; bn <= 128; bn += 64) {
        const int64_t nt = (T + bn - 1) / bn, tiles = mtiles * nt;
        for (int S = 1; S <= 8; ++S) {
            const int64_t kbs = (nkb + S - 1) / S;
            if (S > 1 && (kbs < 4 || (S - 1) * kbs >= nkb || tiles * 2 > kInt8MaxTickets || tiles >= pairs)) break;
            const double block = bn == 64 ? 300 : 2.2 * bn, drain = 1500 + 10.0 * bn;
            const double cost = (double)((tiles * S + pairs - 1) / pairs) * ((double)kbs * block + drain) +
                                (S > 1 ? 1500.0 + 12.0 * bn * S : 0.0);
            if (best.bn == 0 || cost < least) {
                least = cost;
                best.bn = bn;
                best.S = S;
                best.kbs = (int)kbs;
                best.tiles = tiles;
                best.slot_bytes = S > 1 ? (size_t)tiles * 2 * (S + (r > 0 ? 1 : 0)) * bn * kI8Rows * 4 : 0;
            }
        }
    }
    return best;
}

template <int BN>
static cudaError_t launch_int8_gemm_t(const I8GemmArgs& a, int pairs, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute((const void*)int8_gemm_kernel<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         I8Tile<BN>::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * pairs));
    cfg.blockDim = dim3(kI8Threads);
    cfg.dynamicSmemBytes = I8Tile<BN>::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    void* args[] = {(void*)&a};
    return cudaLaunchKernelExC(&cfg, (const void*)int8_gemm_kernel<BN>, args);
}

cudaError_t launch_int8_gemm(const Int8ModuleView* mods, int m, int d, int64_t T, int r, const int8_t* xq,
                             const float* xs, const uint16_t* R, unsigned int* tickets, void* slots,
                             const I8GemmPlan& p, int num_sms, cudaStream_t st) {
    I8GemmArgs a;
    std::memset(&a, 0, sizeof(a));
    const uint32_t half = (uint32_t)(p.bn / 2);
    bool ok = make_map(&a.tmX, CU_TENSOR_MAP_DATA_TYPE_UINT8, xq, (uint64_t)d, (uint64_t)T, (uint64_t)d, kI8Block, half,
                       CU_TENSOR_MAP_SWIZZLE_128B);
    if (r > 0)
        ok = ok && make_map(&a.tmR, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, R, (uint64_t)r, (uint64_t)T, (uint64_t)r * 2, 64, half,
                            CU_TENSOR_MAP_SWIZZLE_128B);
    int mt = 0;
    for (int i = 0; i < m && ok; ++i) {
        const Int8ModuleView& v = mods[i];
        ok = make_map(&a.tmW[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, v.q, (uint64_t)d, (uint64_t)v.O, (uint64_t)d, kI8Block,
                      kI8Rows, CU_TENSOR_MAP_SWIZZLE_128B);
        const bool has_A = r > 0 && v.A;
        if (has_A)
            ok = ok && make_map(&a.tmA[i], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, v.A, (uint64_t)r, (uint64_t)v.O, (uint64_t)r * 2,
                                64, kI8Rows, CU_TENSOR_MAP_SWIZZLE_128B);
        ok = ok && make_map(&a.tmY[i], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, v.Y, (uint64_t)v.O, (uint64_t)T,
                            (uint64_t)v.ldY * 2, kI8Rows, kI8Chunk, CU_TENSOR_MAP_SWIZZLE_NONE);
        a.mod[i] = {v.s, (int)v.O, mt, has_A ? 1 : 0};
        mt += (int)((v.O + 2 * kI8Rows - 1) / (2 * kI8Rows));
    }
    if (!ok) return cudaErrorInvalidValue;
    a.xs = xs;
    a.m = m;
    a.d = d;
    a.T = (int)T;
    a.r = r;
    a.ntiles_n = (int)((T + p.bn - 1) / p.bn);
    a.nunits = (int)(p.tiles * p.S);
    a.S = p.S;
    a.kbs = p.kbs;
    a.slots = static_cast<int4*>(slots);
    a.tickets = tickets;
    a.status = device_status_ptr();
    const int most = gemm_max_pairs(num_sms), pairs = a.nunits < most ? a.nunits : most;
    return p.bn == 64 ? launch_int8_gemm_t<64>(a, pairs, st) : launch_int8_gemm_t<128>(a, pairs, st);
}

}  // namespace glowq
