// int8_gemm.cu -- W8A8 for T > 16 on the 5th-generation tensor cores:
// tcgen05.mma kind::i8 on CTA pairs, int32 accumulators in TMEM.
//
//   y[t][o] = s_t s_o sum_k c[t][k] q[o][k] + sum_j R[t][j] A[o][j]
//
// A cluster of two CTAs computes 256 rows of W x BN tokens: CTA p stages rows
// [128 p, +128) of the codes and half of the tokens' codes (128-byte rows, one
// swizzle atom, by TMA), the leader's MMA thread issues M = 256, N = BN, K = 32
// per step, and each CTA's TMEM receives the int32 sums of its 128 rows, double
// buffered so that a tile's drain overlaps the next tile's products.  A k-block
// of 128 (four steps) takes 565-610 clocks for every BN from 64 to 256 (the
// rows of W set the pace), so BN is the widest that T fills.
//
// Whole tiles: the epilogue turns the sums into s_t s_o sum in fp32 in place,
// the correction's K = 64 slabs of fp16 (A_i and R by TMA, zero beyond r) are
// added to them by the tensor core in the middle of the next tile's products,
// and the epilogue stores y, rounded once.
// Split tiles: what does not make a full round of tiles for every pair (all of
// it when T is small) is one run of k-blocks cut evenly among the pairs, so
// that each streams the same share of W; every segment of a tile stores its
// sums, and int8_join_kernel adds a tile's segments (integers: exact in any
// order), the correction by warp MMA, and stores y.
#include <cstring>
#include <type_traits>

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
constexpr int kI8MaxStages = 9;

template <int BN>
struct I8Tile {
    static constexpr int kHalf = BN / 2;
    static constexpr int kXBytes = kHalf * kI8Block;
    static constexpr int kStageBytes = kI8WBytes + kXBytes;
    static constexpr int kStages = BN == 256 ? 6 : BN == 192 ? 7 : BN == 128 ? 8 : 9;
    static constexpr int kCols = BN == 64 ? 128 : BN == 128 ? 256 : 512;   // two accumulators, a power of two
    static constexpr int kSmem = kStages * kStageBytes + 2 * kI8EpiBytes + 2 * BN * 4 + 512 + 1024;
    static_assert(BN % 64 == 0 && BN <= 256, "MMA N and TMEM columns");
    static_assert(kStages <= kI8MaxStages && kSmem <= kI8SmemMax, "shared memory per CTA");
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
    int ntiles_n;
    I8Split split;
    int* slots;                            // [pair][segment][2 CTAs][BN tokens][128 rows]
    unsigned int* status;
};

struct __align__(8) I8Barriers {
    uint64_t full[kI8MaxStages];   // per CTA: its TMA bytes landed
    uint64_t ready[kI8MaxStages];  // leader: both CTAs' bytes landed (one arrival from each)
    uint64_t empty[kI8MaxStages];  // per CTA: the pair's MMAs that read the stage completed
    uint64_t acc_full[2];          // per CTA: sums complete
    uint64_t conv[2];              // leader: both CTAs turned them into fp32 (one arrival per epilogue warp)
    uint64_t slab_full[2];         // per CTA: correction added
    uint64_t acc_empty[2];         // leader: both CTAs drained them (one arrival per epilogue warp)
    uint32_t tmem_base;
};

// Instruction descriptor, kind::i8: signed int8 A and B, int32 accumulator, both K-major, shape M x N.
__host__ __device__ constexpr uint32_t i8_idesc(int M, int N) {
    return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

struct I8Unit {
    int mi, m0, n0;
    int kb0, nkb, nslab;
    int slot;            // slot of a segment, -1: a whole tile
};
__device__ __forceinline__ I8Unit i8_unit(const I8GemmArgs& a, int bn, int tile, int kb0, int nkb, int slot) {
    I8Unit c;
    const int mt = tile / a.ntiles_n, nt = tile - mt * a.ntiles_n;
    c.mi = 0;
    for (int i = 1; i < a.m; ++i)
        if (mt >= a.mod[i].mtile_begin) c.mi = i;
    c.m0 = (mt - a.mod[c.mi].mtile_begin) * 2 * kI8Rows;
    c.n0 = nt * bn;
    c.kb0 = kb0;
    c.nkb = nkb;
    c.slot = slot;
    c.nslab = (slot < 0 && a.r > 0 && a.mod[c.mi].has_A) ? (a.r + 63) / 64 : 0;
    return c;
}
// The stages of a pair in order, the same for every role: the k-blocks of each
// unit, and the slabs of the unit before it in their midst (its sums are turned
// to fp32 meanwhile, and its buffer is drained before the unit after needs it).
//   begin(unit, n), block(unit, n, i), end(unit, n), slab(unit, n, j); n: units so far
template <class Begin, class Block, class End, class Slab>
__device__ __forceinline__ void i8_walk(const I8GemmArgs& a, int bn, int pair, Begin begin, Block block, End end, Slab slab) {
    I8Unit prev;
    prev.nslab = 0;
    int n = 0, round = 0, seg = 0;
    int64_t pos = i8_share(a.split, pair);
    const int64_t stop = i8_share(a.split, pair + 1);
    while (true) {
        I8Unit c;
        if (round < a.split.rounds) {
            const int64_t tile = (int64_t)round * a.split.pairs + pair;
            ++round;
            if (tile >= a.split.whole) continue;
            c = i8_unit(a, bn, (int)tile, 0, a.split.nkb, -1);
        } else if (pos < stop) {
            const int t = (int)(pos / a.split.nkb), kb0 = (int)(pos - (int64_t)t * a.split.nkb);
            const int nkb = (int)min((int64_t)(a.split.nkb - kb0), stop - pos);
            pos += nkb;
            c = i8_unit(a, bn, a.split.rounds * a.split.pairs + t, kb0, nkb, pair * a.split.segments + seg);
            ++seg;
        } else {
            break;
        }
        begin(c, n);
        const int mid = min(8, (c.nkb + 1) / 2);
        for (int i = 0; i < c.nkb; ++i) {
            block(c, n, i);
            if (i + 1 == mid)
                for (int j = 0; j < prev.nslab; ++j) slab(prev, n - 1, j);
        }
        end(c, n);
        prev = c;
        ++n;
    }
    for (int j = 0; j < prev.nslab; ++j) slab(prev, n - 1, j);
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
    const int pair = (int)cluster_id_x();
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
            mbar_init(&bars->conv[b], 8);
            mbar_init(&bars->slab_full[b], 1);
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
        if (lane == 0) {
            bool ok = true;
            int g = 0, early = 0;
            auto at = [&](int g) { return smem_u32(sm + (g % kStages) * TL::kStageBytes); };
            auto load_w = [&](const I8Unit& c, int i, int g) {
                mbar_arrive_expect_tx(&bars->full[g % kStages], TL::kStageBytes);
                tma_load_2d(at(g), &a.tmW[c.mi], &bars->full[g % kStages], (c.kb0 + i) * kI8Block, c.m0 + row_off);
            };
            auto room = [&]() {
                if (g >= kStages && ok) ok = mbar_wait(&bars->empty[g % kStages], ((g / kStages) - 1) & 1, a.status);
            };
            i8_walk(
                a, BN, pair,
                [&](const I8Unit& c, int n) {
                    if (n > 0) return;
                    // the codes of W are static: the first of them are fetched before the
                    // kernels that quantise X and compute R are known to be complete
                    early = min(kStages, c.nkb);
                    for (int i = 0; i < early; ++i) load_w(c, i, i);
                    pdl_wait();
                },
                [&](const I8Unit& c, int n, int i) {
                    if (g >= early) {
                        room();
                        load_w(c, i, g);
                    }
                    tma_load_2d(at(g) + kI8WBytes, &a.tmX, &bars->full[g % kStages], (c.kb0 + i) * kI8Block, c.n0 + tok_off);
                    ++g;
                },
                [&](const I8Unit&, int) {},
                [&](const I8Unit& c, int n, int j) {
                    room();
                    mbar_arrive_expect_tx(&bars->full[g % kStages], TL::kStageBytes);
                    tma_load_2d(at(g), &a.tmA[c.mi], &bars->full[g % kStages], j * 64, c.m0 + row_off);
                    tma_load_2d(at(g) + kI8WBytes, &a.tmR, &bars->full[g % kStages], j * 64, c.n0 + tok_off);
                    ++g;
                });
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
            auto forward = [&]() {
                if (ok) ok = mbar_wait(&bars->full[g % kStages], (g / kStages) & 1, a.status);
                mbar_arrive_remote(cluster_addr(&bars->ready[g % kStages], 0));
                ++g;
            };
            i8_walk(
                a, BN, pair, [&](const I8Unit&, int) {}, [&](const I8Unit&, int, int) { forward(); },
                [&](const I8Unit&, int) {}, [&](const I8Unit&, int, int) { forward(); });
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
            int s = 0;
            uint32_t ph = 0, convs[2] = {0, 0};
            pdl_wait();
            auto stage = [&](auto integer, uint32_t acc, uint32_t accumulate) {
                if (!next_ready && ok) ok = mbar_wait_cluster(&bars->ready[s], ph, a.status);
                tc_fence_after();
                const int sn = (s + 1 == kStages) ? 0 : s + 1;
                const uint32_t phn = (s + 1 == kStages) ? (ph ^ 1u) : ph;
                constexpr bool kInt = decltype(integer)::value;
                next_ready = i8_stage_mma<kInt>(acc, wdesc + (uint64_t)s * kStageDesc, xdesc + (uint64_t)s * kStageDesc,
                                                kInt ? i8_idesc(2 * kI8Rows, BN) : f16_idesc(2 * kI8Rows, BN), accumulate,
                                                empty_l + 8u * (uint32_t)s, empty_p + 8u * (uint32_t)s,
                                                ready0 + 8u * (uint32_t)sn, phn) != 0;
                s = sn;
                ph = phn;
            };
            int units = 0;
            i8_walk(
                a, BN, pair,
                [&](const I8Unit&, int n) {
                    if (n >= 2 && ok) ok = mbar_wait_cluster(&bars->acc_empty[n & 1], ((n >> 1) - 1) & 1, a.status);
                    tc_fence_after();
                    units = n + 1;
                },
                [&](const I8Unit&, int n, int i) {
                    stage(std::integral_constant<bool, true>{}, tmem + (uint32_t)((n & 1) * BN), i > 0 ? 1u : 0u);
                },
                [&](const I8Unit&, int n) {
                    umma_commit_pair(smem_u32(&bars->acc_full[n & 1]));
                    umma_commit_pair(cluster_addr(&bars->acc_full[n & 1], 1));
                },
                [&](const I8Unit& c, int n, int j) {
                    const int b = n & 1;
                    if (j == 0) {
                        if (ok) ok = mbar_wait_cluster(&bars->conv[b], convs[b] & 1, a.status);
                        ++convs[b];
                    }
                    stage(std::integral_constant<bool, false>{}, tmem + (uint32_t)(b * BN), 1u);
                    if (j + 1 == c.nslab) {
                        umma_commit_pair(smem_u32(&bars->slab_full[b]));
                        umma_commit_pair(cluster_addr(&bars->slab_full[b], 1));
                    }
                });
            for (int n = (units > 2 ? units - 2 : 0); n < units && ok; ++n)
                ok = mbar_wait_cluster(&bars->acc_empty[n & 1], (n >> 1) & 1, a.status);
        }
    } else if (warp >= 4) {
        // ---------------- epilogue (warps 4..7, both CTAs), one thread per row ----------------
        const int quarter = warp & 3, row = quarter * 32 + lane, et = threadIdx.x - 128;
        const bool leader = et == 0;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        bool ok = true;
        int chunk = 0;
        uint32_t slabs[2] = {0, 0};
        pdl_wait();                                       // the token scales are complete
        i8_walk(
            a, BN, pair, [&](const I8Unit&, int) {}, [&](const I8Unit&, int, int) {},
            [&](const I8Unit& c, int n) {
                const int buf = n & 1;
                const uint32_t acc = tmem + lanes + (uint32_t)(buf * BN);
                if (c.slot >= 0) {
                    // a segment of a split tile: its sums to its slot
                    if (ok) ok = mbar_wait(&bars->acc_full[buf], (n >> 1) & 1, a.status);
                    tc_fence_after();
                    int* dst = a.slots + ((int64_t)c.slot * 2 + crank) * (BN * kI8Rows) + row;
                    const int ntok = min(BN, a.T - c.n0);
#pragma unroll 1
                    for (int ch = 0; ch < BN / kI8Chunk; ++ch) {
                        uint32_t v[32];
                        tmem_ld32(acc + ch * kI8Chunk, v);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (ch * kI8Chunk + j < ntok) __stcg(dst + (ch * kI8Chunk + j) * kI8Rows, (int)v[j]);
                    }
                } else {
                    const int orow = c.m0 + row_off + row;
                    const float so = orow < a.mod[c.mi].O ? __ldg(a.mod[c.mi].s + orow) : 0.f;
                    float* ts = tok + buf * BN;           // (its last readers passed the previous unit's first barrier)
                    for (int i = et; i < BN; i += 128) ts[i] = c.n0 + i < a.T ? ldcg_f32(a.xs + c.n0 + i) : 0.f;
                    if (ok) ok = mbar_wait(&bars->acc_full[buf], (n >> 1) & 1, a.status);
                    tc_fence_after();
                    named_barrier_sync(1, 128);           // token scales staged
                    if (c.nslab > 0) {
#pragma unroll 1
                        for (int ch = 0; ch < BN / kI8Chunk; ++ch) {
                            uint32_t v[32];
                            tmem_ld32(acc + ch * kI8Chunk, v);
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                v[j] = __float_as_uint((float)(int)v[j] * ts[ch * kI8Chunk + j] * so);
                            tmem_st32(acc + ch * kI8Chunk, v);
                        }
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_remote(cluster_addr(&bars->conv[buf], 0));
                        if (ok) ok = mbar_wait(&bars->slab_full[buf], slabs[buf] & 1, a.status);
                        ++slabs[buf];
                        tc_fence_after();
                    }
#pragma unroll 1
                    for (int ch = 0; ch < BN / kI8Chunk; ++ch) {
                        const int o0 = c.m0 + row_off, t0 = c.n0 + ch * kI8Chunk;
                        if (t0 >= a.T) break;
                        uint32_t v[32];
                        tmem_ld32(acc + ch * kI8Chunk, v);
                        unsigned char* sb = epi + (chunk & 1) * kI8EpiBytes;
                        ++chunk;
                        if (leader) bulk_wait_read<1>();
                        named_barrier_sync(1, 128);
                        __half* col = reinterpret_cast<__half*>(sb) + row;
                        if (c.nslab > 0) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) col[j * kI8Rows] = __float2half_rn(__uint_as_float(v[j]));
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                col[j * kI8Rows] = __float2half_rn((float)(int)v[j] * ts[ch * kI8Chunk + j] * so);
                        }
                        fence_proxy_async_smem();
                        named_barrier_sync(1, 128);
                        if (leader) {
                            if (o0 < a.mod[c.mi].O) tma_store_2d(&a.tmY[c.mi], smem_u32(sb), o0, t0);
                            bulk_commit();
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(cluster_addr(&bars->acc_empty[buf], 0));
            },
            [&](const I8Unit&, int, int) {});
        if (leader) bulk_wait_all();
    }
    pdl_wait();                                           // every thread: this grid's end implies the preceding ones'
    tc_fence_before();
    __syncwarp();
    cluster_sync_all();                                   // no arrivals or MMA reads into either CTA remain
    if (warp == 1) tmem_dealloc_pair(tmem, TL::kCols);
}

// ---------------------------------------------------------------------------
// Split tiles: one block per 128 rows x 32 tokens of a tile.  A warp has 16
// rows: lane (g, t) the rows g and g + 8 of tokens 2 t, 2 t + 1 of each 8.
// ---------------------------------------------------------------------------
struct I8JoinModule {
    const float* s;
    const __half* A;
    __half* Y;
    int64_t ldY;
    int O, mtile_begin;
};
struct I8JoinArgs {
    I8JoinModule mod[GLOWQ_MAX_MODULES];
    const float* xs;
    const __half* R;
    const int* slots;
    I8Split split;
    int m, T, r, bn, ntiles_n;
};

__global__ void __launch_bounds__(256) int8_join_kernel(const __grid_constant__ I8JoinArgs a) {
    pdl_launch_dependents();
    const int chunks = a.bn / 32;
    const int ch = blockIdx.x % chunks, half = (blockIdx.x / chunks) & 1, rel = blockIdx.x / chunks / 2;
    const int tile = a.split.rounds * a.split.pairs + rel;
    const int mt = tile / a.ntiles_n, nt = tile - mt * a.ntiles_n;
    int mi = 0;
    for (int i = 1; i < a.m; ++i)
        if (mt >= a.mod[i].mtile_begin) mi = i;
    const I8JoinModule& md = a.mod[mi];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int wrow = warp * 16, row0 = (mt - md.mtile_begin) * 2 * kI8Rows + half * kI8Rows + wrow;
    const int t0 = nt * a.bn + ch * 32;
    if (t0 >= a.T || row0 >= md.O) {                      // (O % 16 == 0: a warp's rows are all there or none)
        pdl_wait();
        return;
    }
    // A and the scales are static; R, the sums and the token scales come from the preceding kernels
    const float s0 = __ldg(md.s + row0 + g), s1 = __ldg(md.s + row0 + g + 8);
    const bool corrects = a.r > 0 && md.A;
    uint4 af[4] = {};
    auto load_a = [&](int j0) {
        const __half* A = md.A + (int64_t)(row0 + g) * a.r + j0 + 16 * t;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            af[p] = af[2 + p] = make_uint4(0, 0, 0, 0);
            if (j0 + 16 * t + 8 * p < a.r) {
                af[p] = ldg_128(A + 8 * p);
                af[2 + p] = ldg_128(A + 8 * p + (int64_t)8 * a.r);
            }
        }
    };
    if (corrects) load_a(0);
    pdl_wait();
    // the segments that hold the tile's k-blocks [rel nkb, (rel + 1) nkb): pairs p0 .. p1
    const int64_t lo = (int64_t)rel * a.split.nkb, hi = lo + a.split.nkb;
    int p = (int)(lo * a.split.pairs / a.split.blocks);
    while (i8_share(a.split, p + 1) <= lo) ++p;
    while (i8_share(a.split, p) > lo) --p;
    int v[4][4] = {};
    for (; p < a.split.pairs && i8_share(a.split, p) < hi; ++p) {
        const int64_t begin = i8_share(a.split, p);
        if (begin == i8_share(a.split, p + 1)) continue;  // no share (fewer blocks than pairs)
        const int seg = (int)(rel - begin / a.split.nkb); // the pair's segments are one per tile, in order
        const int* src = a.slots + (((int64_t)p * a.split.segments + seg) * 2 + half) * ((int64_t)a.bn * kI8Rows) +
                         (int64_t)ch * 32 * kI8Rows + wrow + g;
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int tok = n * 8 + 2 * t + e;
                if (t0 + tok < a.T) {
                    v[n][e] += __ldcg(src + tok * kI8Rows);
                    v[n][2 + e] += __ldcg(src + tok * kI8Rows + 8);
                }
            }
    }
    float c[4][4] = {};
    if (corrects) {
        for (int j0 = 0; j0 < a.r; j0 += 64) {
            if (j0 > 0) load_a(j0);
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const int tok = t0 + n * 8 + g;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int j = j0 + 16 * t + 8 * q;
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (tok < a.T && j < a.r) x = ldcg_128(a.R + (int64_t)tok * a.r + j);
                    const uint32_t a1[4] = {af[q].x, af[2 + q].x, af[q].y, af[2 + q].y}, b1[2] = {x.x, x.y};
                    const uint32_t a2[4] = {af[q].z, af[2 + q].z, af[q].w, af[2 + q].w}, b2[2] = {x.z, x.w};
                    mma_16816(c[n], a1, b1);
                    mma_16816(c[n], a2, b2);
                }
            }
        }
    }
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int tok = t0 + n * 8 + 2 * t + e;
            if (tok < a.T) {
                const float st = ldcg_f32(a.xs + tok);
                __half* y = md.Y + (int64_t)tok * md.ldY + row0 + g;
                y[0] = __float2half_rn(fmaf((float)v[n][e] * st, s0, c[n][e]));
                y[8] = __float2half_rn(fmaf((float)v[n][2 + e] * st, s1, c[n][2 + e]));
            }
        }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// Token width: the fewest token tiles, then the narrowest that holds T in them.
// Whole rounds of tiles for every pair, and the rest split, unless a last round
// of whole tiles ends sooner: in clocks, a k-block 600, a split the stores of
// its sums and the join (about 2 us, and the sums' way at 5 TB/s).
I8GemmPlan plan_int8_gemm(int64_t T, int64_t d, int64_t mtiles, int num_sms) {
    I8GemmPlan p;
    const int64_t pairs = gemm_max_pairs(num_sms), nkb = d / kI8Block;
    const int64_t nt = (T + 255) / 256;
    p.bn = (int)(((T + nt - 1) / nt + 63) / 64 * 64);
    const int64_t tiles = mtiles * nt;
    int64_t rounds = tiles / pairs, rest = tiles - rounds * pairs;
    const double blocks = (double)rest * nkb;
    const double split = blocks / pairs * 600 + 4000 + (double)rest * 256 * p.bn * 8 / 2600.0;
    p.split.pairs = (int)(tiles < pairs && rest > 0 && nkb * 600.0 < split ? tiles : pairs);
    if (rest > 0 && nkb * 600.0 < split) {
        // the last round is one of whole tiles: pairs without a tile in it have none
        p.split.whole = tiles;
        rest = 0;
        rounds = (tiles + p.split.pairs - 1) / p.split.pairs;
    } else {
        p.split.whole = rounds * pairs;
    }
    p.split.rounds = (int)rounds;
    p.split.nkb = (int)nkb;
    p.split.blocks = rest * nkb;
    p.split.segments = (int)((p.split.blocks + pairs - 1) / pairs / nkb + 2);
    p.rest = rest;
    p.slot_bytes = rest > 0 ? (size_t)pairs * p.split.segments * 2 * kI8Rows * p.bn * 4 : 0;
    return p;
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
                             const float* xs, const uint16_t* R, int* slots, const I8GemmPlan& p, cudaStream_t st) {
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
    a.split = p.split;
    a.slots = slots;
    a.status = device_status_ptr();
    const int pairs = p.split.pairs;
    cudaError_t e = p.bn == 64    ? launch_int8_gemm_t<64>(a, pairs, st)
                    : p.bn == 128 ? launch_int8_gemm_t<128>(a, pairs, st)
                    : p.bn == 192 ? launch_int8_gemm_t<192>(a, pairs, st)
                                  : launch_int8_gemm_t<256>(a, pairs, st);
    if (e != cudaSuccess || p.rest == 0) return e;
    I8JoinArgs j = {};
    for (int i = 0; i < m; ++i)
        j.mod[i] = {mods[i].s, r > 0 ? reinterpret_cast<const __half*>(mods[i].A) : nullptr, reinterpret_cast<__half*>(mods[i].Y),
                    mods[i].ldY, (int)mods[i].O, a.mod[i].mtile_begin};
    j.xs = xs;
    j.R = reinterpret_cast<const __half*>(R);
    j.slots = slots;
    j.split = p.split;
    j.m = m;
    j.T = (int)T;
    j.r = r;
    j.bn = p.bn;
    j.ntiles_n = a.ntiles_n;
    void* args[] = {(void*)&j};
    return launch_pdl((const void*)int8_join_kernel, (unsigned)(p.rest * 2 * (p.bn / 32)), 256, 0, st, args);
}

}  // namespace glowq
