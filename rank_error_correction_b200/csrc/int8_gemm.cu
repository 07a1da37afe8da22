// int8_gemm.cu -- W8A8 for T > 16 on the 5th-generation tensor cores:
// tcgen05.mma kind::i8 on CTA pairs, int32 accumulators in TMEM.
//
//   y[t][o] = s_t s_o sum_k c[t][k] q[o][k] + sum_j R[t][j] A[o][j]
//
// A cluster of two CTAs computes 256 rows of W x BN tokens: CTA p stages rows
// [128 p, +128) of the codes and half of the tokens' codes (128-byte rows, one
// swizzle atom, by TMA), the leader's MMA thread issues M = 256, N = BN, K = 32
// per step, and each CTA's TMEM receives the int32 sums of its 128 rows, double
// buffered so that a tile's drain overlaps the next tile's products.  BN is as
// wide as T fills, up to 256, where a k-block of 128 (four steps) takes the
// tensor cores 512 clocks: 3.09 POPS measured at T = 2048, d = O = 16384.
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
constexpr int kI8Threads = 192;          // producer, MMA, 4 epilogue warps
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
    unsigned int* counters;                // tokens quantised, blocks done (internal.cuh)
    unsigned int* status;
};

struct __align__(8) I8Barriers {
    uint64_t full[kI8MaxStages];   // leader: both CTAs' TMA bytes landed
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
    int pos = i8_share(a.split, pair);
    const int stop = i8_share(a.split, pair + 1);
    while (true) {
        I8Unit c;
        if (round < a.split.rounds) {
            const int64_t tile = (int64_t)round * a.split.pairs + pair;
            ++round;
            if (tile >= a.split.whole) continue;
            c = i8_unit(a, bn, (int)tile, 0, a.split.nkb, -1);
        } else if (pos < stop) {
            const int t = pos / a.split.nkb, kb0 = pos - t * a.split.nkb;
            const int nkb = min(a.split.nkb - kb0, stop - pos);
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

// Four MMAs of one stage (32 bytes of k each) and the commit that frees it in
// both CTAs, issued by one lane of a warp that runs the loop as a whole: the
// descriptors are then warp-uniform values.  (Inside an `if (lane == 0)` each
// MMA took about 140 clocks to issue whatever its N, most of it moving
// descriptors into uniform registers.)
template <bool INT>
__device__ __forceinline__ void i8_stage_mma(uint32_t dacc, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate, uint32_t empty) {
#define GLOWQ_STAGE_MMA(KIND)                                                                             \
    asm volatile(                                                                                         \
        "{\n\t.reg .pred pe, pa, pt;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t.reg .b16 both;\n\t"      \
        "elect.sync _|pe, 0xffffffff;\n\t"                                                               \
        "setp.ne.b32 pa, %2, 0;\n\t"                                                                     \
        "setp.eq.b32 pt, %2, %2;\n\t"                                                                    \
        "mov.b16 both, 3;\n\t"                                                                           \
        "add.s64 a1, %4, 2;\n\tadd.s64 a2, %4, 4;\n\tadd.s64 a3, %4, 6;\n\t"                           \
        "add.s64 b1, %5, 2;\n\tadd.s64 b2, %5, 4;\n\tadd.s64 b3, %5, 6;\n\t"                           \
        "@pe tcgen05.mma.cta_group::2.kind::" KIND " [%0], %4, %5, %1, pa;\n\t"                          \
        "@pe tcgen05.mma.cta_group::2.kind::" KIND " [%0], a1, b1, %1, pt;\n\t"                          \
        "@pe tcgen05.mma.cta_group::2.kind::" KIND " [%0], a2, b2, %1, pt;\n\t"                          \
        "@pe tcgen05.mma.cta_group::2.kind::" KIND " [%0], a3, b3, %1, pt;\n\t"                          \
        "@pe tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%3], both;\n\t}" \
        ::"r"(dacc), "r"(idesc), "r"(accumulate), "r"(empty), "l"(adesc), "l"(bdesc)                      \
        : "memory")
    if constexpr (INT) {
        GLOWQ_STAGE_MMA("i8");
    } else {
        GLOWQ_STAGE_MMA("f16");
    }
#undef GLOWQ_STAGE_MMA
}
// Arrive on the barrier at this offset in both CTAs of the pair once the MMAs issued so far complete (one lane).
__device__ __forceinline__ void i8_commit_both(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred pe;\n\t.reg .b16 both;\n\t"
        "elect.sync _|pe, 0xffffffff;\n\tmov.b16 both, 3;\n\t"
        "@pe tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], both;\n\t}" ::"r"(bar)
        : "memory");
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
        // ---------------- producer (both CTAs, the whole warp) ----------------
        bool ok = true, r_ready = false;
        int g = 0, s = 0, early = 0;                       // stages so far, ring stage, stages whose W is fetched ahead
        uint32_t ph = 1;                                   // parity of empty[s] that frees the stage (the first use: free)
        const uint32_t base = smem_u32(sm), empty0 = smem_u32(&bars->empty[0]), full0 = smem_u32(&bars->full[0]);
        const uint32_t lead0 = cluster_addr(&bars->full[0], 0);
        // stage `st` is free: announce both CTAs' bytes on the leader's barrier
        auto announce = [&](int st) {
            if (crank == 0) expect_tx_elect(full0 + 8u * (uint32_t)st, 2 * TL::kStageBytes);
        };
        auto load = [&](uint32_t off, const CUtensorMap* map, int st, int x, int y) {
            tma_load_2d_pair(base + (uint32_t)(st * TL::kStageBytes) + off, map, lead0 + 8u * (uint32_t)st, x, y);
        };
        auto room = [&]() {
            if (g >= kStages && ok) ok = mbar_wait_warp(empty0 + 8u * (uint32_t)s, ph, a.status);
        };
        auto advance = [&]() {
            ++g;
            if (++s == kStages) {
                s = 0;
                ph ^= 1u;
            }
        };
        i8_walk(
            a, BN, pair,
            [&](const I8Unit& c, int n) {
                if (n > 0) return;
                // the codes of W are static: the first of them are fetched while X is quantised
                early = min(kStages, c.nkb);
                for (int i = 0; i < early; ++i) {
                    announce(i);
                    load(0, &a.tmW[c.mi], i, (c.kb0 + i) * kI8Block, c.m0 + row_off);
                }
                wait_ready(a.counters, (unsigned)a.T);
                fence_proxy_async_all();
            },
            [&](const I8Unit& c, int n, int i) {
                if (g >= early) {
                    room();
                    announce(s);
                    load(0, &a.tmW[c.mi], s, (c.kb0 + i) * kI8Block, c.m0 + row_off);
                }
                load(kI8WBytes, &a.tmX, s, (c.kb0 + i) * kI8Block, c.n0 + tok_off);
                advance();
            },
            [&](const I8Unit&, int) {},
            [&](const I8Unit& c, int n, int j) {
                if (!r_ready) pdl_wait();                  // R is complete
                r_ready = true;
                room();
                announce(s);
                load(0, &a.tmA[c.mi], s, j * 64, c.m0 + row_off);
                load(kI8WBytes, &a.tmR, s, j * 64, c.n0 + tok_off);
                advance();
            });
        // the leader's commits for the last stages land here before this CTA may exit
        for (int p = (g > kStages ? g - kStages : 0); p < g && ok; ++p)
            ok = mbar_wait_warp(empty0 + 8u * (uint32_t)(p % kStages), (uint32_t)(p / kStages) & 1u, a.status);
    } else if (warp == 1) {
        // ---------------- MMA issuer (leader CTA, the whole warp) ----------------
        if (crank == 0) {
            constexpr uint64_t kStageDesc = (uint64_t)(TL::kStageBytes >> 4);
            const uint64_t wdesc = sw128_kmajor_desc(smem_u32(sm));
            const uint64_t xdesc = sw128_kmajor_desc(smem_u32(sm) + kI8WBytes);
            const uint32_t empty0 = smem_u32(&bars->empty[0]), full0 = smem_u32(&bars->full[0]);
            bool ok = true;
            int s = 0, units = 0;
            uint32_t ph = 0, convs = 0;                    // convs: bit b: parity of conv[b]
            wait_ready(a.counters, (unsigned)a.T);         // (the bounded waits below begin when the codes can come)
            auto stage = [&](auto integer, uint32_t acc, uint32_t accumulate) {
                if (ok) ok = mbar_wait_warp(full0 + 8u * (uint32_t)s, ph, a.status);
                tc_fence_after();
                constexpr bool kInt = decltype(integer)::value;
                i8_stage_mma<kInt>(acc, wdesc + (uint64_t)s * kStageDesc, xdesc + (uint64_t)s * kStageDesc,
                                   kInt ? i8_idesc(2 * kI8Rows, BN) : f16_idesc(2 * kI8Rows, BN), accumulate,
                                   empty0 + 8u * (uint32_t)s);
                if (++s == kStages) {
                    s = 0;
                    ph ^= 1u;
                }
            };
            i8_walk(
                a, BN, pair,
                [&](const I8Unit&, int n) {
                    if (n >= 2 && ok) ok = mbar_wait_warp(smem_u32(&bars->acc_empty[n & 1]), ((n >> 1) - 1) & 1, a.status);
                    tc_fence_after();
                    units = n + 1;
                },
                [&](const I8Unit&, int n, int i) {
                    stage(std::integral_constant<bool, true>{}, tmem + (uint32_t)((n & 1) * BN), i > 0 ? 1u : 0u);
                },
                [&](const I8Unit&, int n) { i8_commit_both(smem_u32(&bars->acc_full[n & 1])); },
                [&](const I8Unit& c, int n, int j) {
                    const uint32_t b = (uint32_t)(n & 1);
                    if (j == 0) {
                        if (ok) ok = mbar_wait_warp(smem_u32(&bars->conv[b]), (convs >> b) & 1u, a.status);
                        convs ^= 1u << b;
                    }
                    stage(std::integral_constant<bool, false>{}, tmem + b * BN, 1u);
                    if (j + 1 == c.nslab) i8_commit_both(smem_u32(&bars->slab_full[b]));
                });
            for (int n = (units > 2 ? units - 2 : 0); n < units && ok; ++n)
                ok = mbar_wait_warp(smem_u32(&bars->acc_empty[n & 1]), (n >> 1) & 1, a.status);
        }
    } else {
        // ---------------- epilogue (warps 2..5, both CTAs), one thread per row ----------------
        const int quarter = warp & 3, row = quarter * 32 + lane, et = threadIdx.x - 64;
        const bool leader = et == 0;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        bool ok = true;
        int chunk = 0;
        uint32_t slabs = 0;                               // bit b: parity of slab_full[b]
        wait_ready(a.counters, (unsigned)a.T);            // the token scales are complete
        pdl_wait();                                       // ... and the previous readers of Y and the slots are done
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
                        if (ok) ok = mbar_wait(&bars->slab_full[buf], (slabs >> buf) & 1, a.status);
                        slabs ^= 1u << buf;
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
    if (threadIdx.x == 0) {                               // the last block to end returns the counters to zero
        if (atomicAdd(a.counters + 1, 1u) == gridDim.x - 1) {
            atomicExch(a.counters, 0u);
            atomicExch(a.counters + 1, 0u);
        }
    }
}

// ---------------------------------------------------------------------------
// R = X B^T ahead of the product: a cluster of eight blocks takes 128 tokens,
// block c the c-th eighth of d (tcgen05, M = 128 tokens, N = r, both operands by
// TMA, fp32 in TMEM).  The eight parts meet in distributed shared memory: block
// c adds the parts of tokens 16 c .. + 15 in block order and rounds R to fp16.
// ---------------------------------------------------------------------------
constexpr int kProjParts = 8, kProjThreads = 192, kProjStages = 8;

struct I8ProjArgs {
    CUtensorMap tmX;      // X [T][d] fp16, box {64, 128}, SW128
    CUtensorMap tmB;      // B [r][d] fp16, box {64, rn}, SW128
    __half* R;
    int d, T, r, rn, stages;
    unsigned int* status;
};
__host__ __device__ inline int proj_stage_bytes(int rn) { return 128 * 128 + rn * 128; }
__host__ __device__ inline int proj_pitch(int rn) { return rn + 4; }     // floats
static size_t proj_ring_bytes(int rn, int stages) {
    const size_t ring = (size_t)stages * proj_stage_bytes(rn), sums = (size_t)128 * proj_pitch(rn) * 4;
    return ((ring > sums ? ring : sums) + 1023) / 1024 * 1024;
}

__global__ void __launch_bounds__(kProjThreads, 1) int8_project_kernel(const __grid_constant__ I8ProjArgs a, uint32_t ring_bytes) {
    extern __shared__ __align__(1024) unsigned char raw[];
    unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    struct Bars {
        uint64_t full[kProjStages], empty[kProjStages], acc;
        uint32_t tmem;
    };
    Bars* bars = reinterpret_cast<Bars*>(sm + ring_bytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t part = cluster_ctarank();
    const int t0 = (int)(blockIdx.x / kProjParts) * 128;
    const int nkb = a.d / 64, kb0 = (int)part * nkb / kProjParts, n = (int)(part + 1) * nkb / kProjParts - kb0;
    const int sbytes = proj_stage_bytes(a.rn);
    uint32_t ncols = 32;
    while (ncols < (uint32_t)a.rn) ncols <<= 1;
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], 1);
        }
        mbar_init(&bars->acc, 1);
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(&bars->tmem, ncols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem;
    pdl_wait();                 // X may be produced by the preceding kernel; the previous call's readers of R are done
    pdl_launch_dependents();
    if (warp == 0) {
        bool ok = true;
        for (int i = 0; i < n; ++i) {
            const int s = i % a.stages;
            if (i >= a.stages && ok) ok = mbar_wait_warp(smem_u32(&bars->empty[s]), (uint32_t)(i / a.stages - 1) & 1u, a.status);
            const uint32_t full = smem_u32(&bars->full[s]), dst = smem_u32(sm) + (uint32_t)(s * sbytes);
            expect_tx_elect(full, (uint32_t)sbytes);
            tma_load_2d_elect(dst, &a.tmX, full, (kb0 + i) * 64, t0);
            tma_load_2d_elect(dst + 128 * 128, &a.tmB, full, (kb0 + i) * 64, 0);
        }
    } else if (warp == 1) {
        const uint32_t idesc = f16_idesc(128, a.rn);
        bool ok = true;
        for (int i = 0; i < n; ++i) {
            const int s = i % a.stages;
            if (ok) ok = mbar_wait_warp(smem_u32(&bars->full[s]), (uint32_t)(i / a.stages) & 1u, a.status);
            tc_fence_after();
            const uint64_t ad = sw128_kmajor_desc(smem_u32(sm) + (uint32_t)(s * sbytes));
            umma_f16_stage_elect(tmem, ad, ad + (uint64_t)(128 * 128 / 16), idesc, i > 0 ? 1u : 0u, smem_u32(&bars->empty[s]));
        }
        umma_commit_elect(smem_u32(&bars->acc));
    }
    // the part's sums over the ring (its loads and products are complete): [128 tokens][pitch]
    const int pitch = proj_pitch(a.rn);
    float* sums = reinterpret_cast<float*>(sm);
    if (warp >= 2) {
        const int quarter = warp & 3, row = quarter * 32 + lane;
        mbar_wait(&bars->acc, 0, a.status);
        tc_fence_after();
        for (int c = 0; c < a.rn; c += 32) {
            uint32_t v[32];
            if (n > 0) {
                tmem_ld32(tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)c, v);
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = 0u;
            }
#pragma unroll
            for (int j = 0; j < 32; j += 4)
                if (c + j < a.rn)
                    *reinterpret_cast<uint4*>(sums + row * pitch + c + j) = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync_all();
    const int q4 = a.r / 4;
    for (int i = threadIdx.x; i < 16 * q4; i += kProjThreads) {
        const int row = (int)part * 16 + i / q4, c = i % q4 * 4;
        float4 p[kProjParts];
#pragma unroll
        for (int k = 0; k < kProjParts; ++k) {
            const uint32_t at = cluster_addr(sums + row * pitch + c, (uint32_t)k);
            asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                         : "=f"(p[k].x), "=f"(p[k].y), "=f"(p[k].z), "=f"(p[k].w)
                         : "r"(at)
                         : "memory");
        }
        float4 v = p[0];
#pragma unroll
        for (int k = 1; k < kProjParts; ++k) v.x += p[k].x, v.y += p[k].y, v.z += p[k].z, v.w += p[k].w;
        if (t0 + row < a.T) {
            uint2 o;
            o.x = h2_as_u32(__floats2half2_rn(v.x, v.y));
            o.y = h2_as_u32(__floats2half2_rn(v.z, v.w));
            *reinterpret_cast<uint2*>(a.R + (int64_t)(t0 + row) * a.r + c) = o;
        }
    }
    __syncwarp();
    cluster_sync_all();          // no block's shared memory is read any more
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, ncols);
}

// ---------------------------------------------------------------------------
// Split tiles: one block per 128 rows x 32 tokens of a tile, a warp per 32
// rows.  Lane (g, t) has the rows 4 g .. 4 g + 3 (they are rows g and g + 8 of
// the MMA's two row tiles) of tokens 2 t, 2 t + 1 of each 8, so sums come 16
// bytes and outputs go 8 bytes at a time.
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 128;

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

__global__ void __launch_bounds__(kJoinThreads, 3) int8_join_kernel(const __grid_constant__ I8JoinArgs a) {
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
    const int trow = warp * 32 + 4 * g;                   // this lane's first row within the CTA's 128
    const int row = (mt - md.mtile_begin) * 2 * kI8Rows + half * kI8Rows + trow;
    const int t0 = nt * a.bn + ch * 32;
    // A and the scales are static; R, the sums and the token scales come from the preceding kernels
    const bool there = row < md.O, corrects = a.r > 0 && md.A;      // (O % 16 == 0: four rows are there or none)
    float4 so = make_float4(0.f, 0.f, 0.f, 0.f);
    if (there) so = make_float4(__ldg(md.s + row), __ldg(md.s + row + 1), __ldg(md.s + row + 2), __ldg(md.s + row + 3));
    uint4 af[4][2];
    auto load_a = [&](int j0) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int j = j0 + 16 * t + 8 * p;
                af[i][p] = make_uint4(0, 0, 0, 0);
                if (there && j < a.r) af[i][p] = ldg_128(md.A + (int64_t)(row + i) * a.r + j);
            }
    };
    if (corrects) load_a(0);
    pdl_wait();
    if (t0 >= a.T) return;
    // the segments that hold the tile's k-blocks [rel nkb, (rel + 1) nkb): those of pairs p0 .. p1
    const int nkb = a.split.nkb, lo = rel * nkb, hi = lo + nkb;
    int p = lo * a.split.sharers / a.split.blocks;
    while (i8_share(a.split, p + 1) <= lo) ++p;
    while (i8_share(a.split, p) > lo) --p;
    // R of the first 64 columns and the token scales, in flight beside the sums
    uint4 rx[4][2];
    auto load_r = [&](int j0) {
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int tok = t0 + n * 8 + g, j = j0 + 16 * t + 8 * q;
                rx[n][q] = ldcg_128_if(a.R + (int64_t)tok * a.r + j, tok < a.T && j < a.r);
            }
    };
    if (corrects) load_r(0);
    float st[4][2];
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int tok = t0 + n * 8 + 2 * t + e;
            st[n][e] = ldcg_f32(a.xs + min(tok, a.T - 1));
        }
    int v[4][2][4] = {};
    for (int begin = i8_share(a.split, p); p < a.split.sharers && begin < hi; begin = i8_share(a.split, ++p)) {
        const int seg = rel - begin / nkb;                // the pair's segments are one per tile, in order
        const int* src = a.slots + (((int64_t)p * a.split.segments + seg) * 2 + half) * ((int64_t)a.bn * kI8Rows) +
                         (int64_t)ch * 32 * kI8Rows + trow;
        int4 x[4][2];
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int tok = n * 8 + 2 * t + e;
                const uint4 u = ldcg_128_if(src + tok * kI8Rows, t0 + tok < a.T);
                x[n][e] = make_int4((int)u.x, (int)u.y, (int)u.z, (int)u.w);
            }
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                v[n][e][0] += x[n][e].x;
                v[n][e][1] += x[n][e].y;
                v[n][e][2] += x[n][e].z;
                v[n][e][3] += x[n][e].w;
            }
    }
    float c[2][4][4] = {};
    if (corrects) {
        for (int j0 = 0; j0 < a.r; j0 += 64) {
            if (j0 > 0) {
                load_a(j0);
                load_r(j0);
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const uint4(&x)[2] = rx[n];
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int w = 0; w < 2; ++w) {         // row tiles: rows 4 g, 4 g + 1 and 4 g + 2, 4 g + 3
                        const uint4 &u = af[2 * w][q], &l = af[2 * w + 1][q];
                        const uint32_t a1[4] = {u.x, l.x, u.y, l.y}, b1[2] = {x[q].x, x[q].y};
                        const uint32_t a2[4] = {u.z, l.z, u.w, l.w}, b2[2] = {x[q].z, x[q].w};
                        mma_16816(c[w][n], a1, b1);
                        mma_16816(c[w][n], a2, b2);
                    }
            }
        }
    }
    if (!there) return;
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int tok = t0 + n * 8 + 2 * t + e;
            if (tok < a.T) {
                const float s = st[n][e];
                uint2 y;
                y.x = h2_as_u32(__floats2half2_rn(fmaf((float)v[n][e][0] * s, so.x, c[0][n][e]),
                                                  fmaf((float)v[n][e][1] * s, so.y, c[0][n][2 + e])));
                y.y = h2_as_u32(__floats2half2_rn(fmaf((float)v[n][e][2] * s, so.z, c[1][n][e]),
                                                  fmaf((float)v[n][e][3] * s, so.w, c[1][n][2 + e])));
                *reinterpret_cast<uint2*>(md.Y + (int64_t)tok * md.ldY + row) = y;
            }
        }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
cudaError_t launch_int8_project(const uint16_t* X, const uint16_t* B, int64_t T, int d, int r, uint16_t* R,
                                cudaStream_t st) {
    I8ProjArgs a;
    std::memset(&a, 0, sizeof(a));
    a.rn = (r + 15) / 16 * 16;
    if (!make_map(&a.tmX, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, X, (uint64_t)d, (uint64_t)T, (uint64_t)d * 2, 64, 128,
                  CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map(&a.tmB, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, B, (uint64_t)d, (uint64_t)r, (uint64_t)d * 2, 64, (uint32_t)a.rn,
                  CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    a.R = reinterpret_cast<__half*>(R);
    a.d = d;
    a.T = (int)T;
    a.r = r;
    a.status = device_status_ptr();
    const int most = 104 * 1024 / proj_stage_bytes(a.rn);        // two blocks an SM: 4 stages at r = 64, 2 at r = 256
    a.stages = most > kProjStages ? kProjStages : most;
    uint32_t ring = (uint32_t)proj_ring_bytes(a.rn, a.stages);
    static SmemLimit limit;
    cudaError_t e = limit.raise((const void*)int8_project_kernel, kI8SmemMax);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((T + 127) / 128 * kProjParts));
    cfg.blockDim = dim3(kProjThreads);
    cfg.dynamicSmemBytes = ring + 1024 + 256;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kProjParts;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    void* args[] = {(void*)&a, (void*)&ring};
    return cudaLaunchKernelExC(&cfg, (const void*)int8_project_kernel, args);
}

// Token width: the fewest token tiles, then the narrowest that holds T in them.
// Whole rounds of tiles for every pair, and the rest split, unless a last round
// of whole tiles ends sooner: in clocks, a k-block 600, a split the stores of
// its sums and the join (about 2 us, and the sums' way at 5 TB/s).
I8GemmPlan plan_int8_gemm(int64_t T, int64_t d, int64_t mtiles, int num_sms) {
    I8GemmPlan p;
    const int64_t nkb = d / kI8Block, nt = (T + 255) / 256, tiles = mtiles * nt;
    p.bn = (int)(((T + nt - 1) / nt + 63) / 64 * 64);
    int64_t pairs = gemm_max_pairs(num_sms);
    int64_t rounds = tiles / pairs, rest = tiles - rounds * pairs;
    p.split.whole = rounds * pairs;
    // no share below 8 blocks: the join reads every share of a tile
    int64_t sharers = rest * nkb / 8;
    sharers = sharers < 1 ? 1 : sharers > pairs ? pairs : sharers;
    const double whole = nkb * 600.0;
    const double split = (double)rest * nkb / sharers * 600 + 4000 + (double)rest * 256 * p.bn * 8 / 2600.0;
    if (rest > 0 && whole < split) {
        // the last round is one of whole tiles: pairs without a tile in it have none
        p.split.whole = tiles;
        if (rounds == 0) pairs = tiles;
        ++rounds;
        rest = 0;
    }
    if (rest > 0 && rounds == 0) pairs = sharers;
    p.split.pairs = (int)pairs;
    p.split.sharers = (int)sharers;
    p.split.rounds = (int)rounds;
    p.split.nkb = (int)nkb;
    p.split.blocks = (int)(rest * nkb);
    p.split.segments = (int)((rest * nkb + sharers - 1) / sharers / nkb + 2);
    p.rest = rest;
    p.slot_bytes = rest > 0 ? (size_t)sharers * p.split.segments * 2 * kI8Rows * p.bn * 4 : 0;
    return p;
}

template <int BN>
static cudaError_t launch_int8_gemm_t(const I8GemmArgs& a, int pairs, cudaStream_t st) {
    static SmemLimit limit;
    cudaError_t e = limit.raise((const void*)int8_gemm_kernel<BN>, I8Tile<BN>::kSmem);
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
                             const float* xs, const uint16_t* R, unsigned int* tickets, int* slots, const I8GemmPlan& p,
                             cudaStream_t st) {
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
    a.counters = tickets + kInt8Ready;
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
    return launch_pdl((const void*)int8_join_kernel, (unsigned)(p.rest * 2 * (p.bn / 32)), kJoinThreads, 0, st,
                      args);
}

}  // namespace glowq
