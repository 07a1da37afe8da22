// attention_tc.cu -- attention of many query rows (prefill, chunks) over the
// paged 8-bit cache on the 5th-generation tensor cores; the formulas of
// attention.cu.
//
// A block takes 256 rows (row = new token i and query head gq of the kv head's
// group, i G + gq) of one sequence and kv head, as two tiles of 128 rows that
// share every key and value, over tiles of 128 tokens (two pages):
//   S_t = Q_t K^T       128 x 128 x D, Q and K in shared memory (fp16)
//   P_t = 2^(S_t a - m) in fp16 over S_t's columns of TMEM
//   O_t += P_t V        P from TMEM, V in shared memory
// The four accumulators S_0, S_1, O_0, O_1 fill TMEM at D = 128.  While one
// tile's softmax runs, the tensor cores work on the other's products.
// The cache's layouts are the operands': a row of 64 codes (64 dimensions of a
// key, 64 tokens of a value's dimension) becomes a 128-byte row of fp16 in the
// K-major 128-byte-swizzled layout, so converting is all the staging there is.
// A row's reference is moved only when its maximum has grown by 2^6 or more
// (then O is rescaled in TMEM): weights stay below 2^14.
// Warps: 0-3 and 4-7 softmax of tiles 0 and 1 (a thread per row), 8-11 convert
// pages, 12 issues the MMAs.
// 4096 new tokens of 32 heads of 128: 186 us, 739 TFLOP/s (45 % of the dense
// rate); four chunks of 187 to 821 tokens, 8 kv heads: 104 us.  256 rows and 128
// tokens take 5000 clocks, of which the tensor pipe works 2050, the exponentials
// 2050 and shared memory 2560, and issue slots are 42 % busy: what bounds it is
// how far these overlap.  Slower: scores of a page in two buffers, so that a
// tile's next scores wait for it (198 us: products of 64 columns are bound by the
// reads of Q, 52 clocks for 32 of work); eight converting warps (202 us: 96
// registers); a part of the exponentials as polynomials (202 to 217 us).
#include "internal.cuh"
#include "kvcache.cuh"
#include "tc.cuh"

namespace glowq {

constexpr int kTcRows = 256, kTcTokens = 128, kTcThreads = 512, kTcMeta = 4;
constexpr int kTcLeastTiles = 4, kTcMostShares = 16, kTcMostTickets = 16384, kTcMostPairs = 256;
constexpr float kTcWeightExp = 8.f, kTcSlack = 6.f, kTcApart = 1048576.f;

struct KvTcArgs {
    KvCacheView c;
    KvBatchView b;
    const uint16_t* Q;
    uint16_t* Y;
    int64_t ldQ, ldY;
    float scale_log2;
    int G, rt;               // query heads per kv head, row tiles of the widest sequence
    int S;                   // shares of a unit's tokens, at most
    float* partial;          // [row tile of the batch][kv head][share][D + 2][256 rows]: O by column, base, l
    unsigned int* tickets;   // [unit of the grid], zero between calls
    unsigned int* status;
};

// What a softmax needs of a tile's two pages.
struct KvTcMeta {
    float a[2];              // s_K scale log2(e)
    float lv[2];             // log2 s_V
    float inv[2];            // 1 / s_V
    int valid[2];            // tokens present
};
struct __align__(8) KvTcShared {
    uint64_t q_full, kf[2], ke[2], vf[2], ve[2], s_full[2], p_full[2], o_done[2];
    uint64_t codes[2];                   // the staged codes of K, of V
    KvTcMeta meta[kTcMeta];
    unsigned int tail_max, tail_poison[2];
    int last;                            // this block joins its unit's shares
    int pair;                            // its row tile and sequence
    uint32_t tmem;
};

template <int D>
struct KvTc {
    static constexpr int kPanels = D / 64;
    static constexpr int kQBytes = 128 * D * 2;          // one row tile: panels of [128 rows][128 B]
    static constexpr int kKBytes = kTcTokens * D * 2;    // panels of [128 tokens][128 B]
    static constexpr int kVBytes = 2 * D * 128;          // pages of [D][128 B]
    static constexpr int kCodes = 2 * kKvPage * D;       // one tile's K (or V) codes
    static constexpr int kSmem = 2 * kQBytes + 2 * kKBytes + 2 * kVBytes + 2 * kCodes + (int)sizeof(KvTcShared) + 1024;
    static_assert(kSmem <= 232448, "shared memory per block");
};

__device__ __forceinline__ void tc_cvt_codes(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = w ^ 0x80808080u;
    const __half2 bias = u32_as_h2(0x64806480u);         // 1152
    lo = h2_as_u32(__hsub2(u32_as_h2(__byte_perm(u, 0x64646464u, 0x4140)), bias));
    hi = h2_as_u32(__hsub2(u32_as_h2(__byte_perm(u, 0x64646464u, 0x4342)), bias));
}
__device__ __forceinline__ float tc_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 64 columns of this thread's lane, complete on return (load and wait in one
// statement: a wait of its own would need the registers as operands, and moves them).
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&v)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
        "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
        "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
        "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63"
        "}, [%64];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), 
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), 
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), 
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31]), 
          "=r"(v[32]), "=r"(v[33]), "=r"(v[34]), "=r"(v[35]), "=r"(v[36]), "=r"(v[37]), "=r"(v[38]), "=r"(v[39]), 
          "=r"(v[40]), "=r"(v[41]), "=r"(v[42]), "=r"(v[43]), "=r"(v[44]), "=r"(v[45]), "=r"(v[46]), "=r"(v[47]), 
          "=r"(v[48]), "=r"(v[49]), "=r"(v[50]), "=r"(v[51]), "=r"(v[52]), "=r"(v[53]), "=r"(v[54]), "=r"(v[55]), 
          "=r"(v[56]), "=r"(v[57]), "=r"(v[58]), "=r"(v[59]), "=r"(v[60]), "=r"(v[61]), "=r"(v[62]), "=r"(v[63])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
          "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// One K = 16 step, A in shared memory or in TMEM; issued by one lane of the warp.
__device__ __forceinline__ void umma_ss_elect(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred pe, pa;\n\telect.sync _|pe, 0xffffffff;\n\tsetp.ne.b32 pa, %4, 0;\n\t"
        "@pe tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, pa;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void umma_ts_elect(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred pe, pa;\n\telect.sync _|pe, 0xffffffff;\n\tsetp.ne.b32 pa, %4, 0;\n\t"
        "@pe tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, pa;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// Byte offset of 16-byte chunk c of row r in the swizzled layout.
__device__ __forceinline__ uint32_t sw128(int r, int c) {
    return (uint32_t)((r >> 3) * 1024 + (r & 7) * 128 + ((c ^ (r & 7)) << 4));
}

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1) kv_attention_tc_kernel(const __grid_constant__ KvTcArgs a) {
    using L = KvTc<D>;
    extern __shared__ __align__(1024) unsigned char raw[];
    unsigned char* sq = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    unsigned char* sk = sq + 2 * L::kQBytes;
    unsigned char* sv = sk + 2 * L::kKBytes;
    unsigned char* sc = sv + 2 * L::kVBytes;
    KvTcShared* sh = reinterpret_cast<KvTcShared*>(sc + 2 * L::kCodes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int share = blockIdx.x % a.S, unit = blockIdx.x / a.S, h = unit % a.c.kv_heads;
    int pair = unit / a.c.kv_heads;                                  // (row tile, sequence), the last rows first
    if (threadIdx.x == 0) {
        mbar_init(&sh->q_full, 8);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh->kf[i], 4);
            mbar_init(&sh->ke[i], 1);
            mbar_init(&sh->vf[i], 4);
            mbar_init(&sh->ve[i], 1);
            mbar_init(&sh->s_full[i], 1);
            mbar_init(&sh->p_full[i], 4);
            mbar_init(&sh->o_done[i], 1);
            mbar_init(&sh->codes[i], 1);
        }
        fence_mbar_init();
    }
    pdl_wait();
    const int pairs = a.rt * a.b.n_seq;
    if (a.b.n_seq > 1 && pairs <= kTcMostPairs) {
        // The longest first, whatever the sequences' lengths: the pair of this block's rank (four uneven
        // chunks: 103 us instead of 126).
        int* len = reinterpret_cast<int*>(sk);
        const int i = threadIdx.x;
        int mine = 0, rank = 0;
        if (i < pairs) {
            const KvSeq q = kv_sequence(a.b, i % a.b.n_seq);
            const int first = (a.rt - 1 - i / a.b.n_seq) * kTcRows, n = q.nq * a.G;
            mine = first < n ? max(0, q.start + (min(first + kTcRows, n) - 1) / a.G) / kTcTokens + 1 : 0;
            len[i] = mine;
        }
        __syncthreads();
        if (i < pairs) {
            for (int k = 0; k < pairs; ++k) rank += len[k] > mine || (len[k] == mine && k < i);
            if (rank == pair) sh->pair = i;
        }
        __syncthreads();
        pair = sh->pair;
    }
    const int tile = a.rt - 1 - pair / a.b.n_seq, b = pair % a.b.n_seq;
    const KvSeq s = kv_sequence(a.b, b);
    const int rows = s.nq * a.G, row0 = tile * kTcRows;
    if (!s.ok && threadIdx.x == 0) record_status(a.status, GLOWQ_ERR_INDEX);
    if (row0 >= rows) return;
    // a length that the table or the tails cannot hold: nothing is visible, and the rows are zero
    const bool tailed = s.len % kKvPage != 0;
    const bool bad = s.len > (int64_t)a.b.max_pages * kKvPage || (tailed && (s.slot < 0 || s.slot >= a.c.slots));
    if (bad && threadIdx.x == 0) record_status(a.status, GLOWQ_ERR_INDEX);
    int nt[2];                                                       // token tiles that each row tile sees
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int first = row0 + t * 128, last = min(first + 127, rows - 1);
        const int seen = bad || first >= rows ? 0 : max(0, s.start + last / a.G + 1);
        nt[t] = (seen + kTcTokens - 1) / kTcTokens;
    }
    // this block's share of the token tiles; from here on tiles, pages and positions count from its first
    int nmax = max(nt[0], nt[1]);
    const int per = max((nmax + a.S - 1) / a.S, kTcLeastTiles), shares = max(1, (nmax + per - 1) / per);
    if (share >= shares) return;
    const int ja = share * per;
#pragma unroll
    for (int t = 0; t < 2; ++t) nt[t] = max(0, min(nt[t] - ja, per));
    nmax = max(nt[0], nt[1]);
    if (warp == 12) tmem_alloc(&sh->tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem;                                  // S_0, S_1 (128 columns each), O_0, O_1
    // only now: a kernel that began earlier might take TMEM that a block of this
    // grid still waits for, and wait for this grid's end itself
    pdl_launch_dependents();
    bool ok = true;

    if (warp < 8) {
        // ---------------- softmax: one thread per row ----------------
        const int t = warp >> 2, r = (warp & 3) * 32 + lane, row = row0 + t * 128 + r;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + (uint32_t)(t * 128), to = tmem + lanes + (uint32_t)(256 + t * 128);
        const bool there = row < rows;
        const int tok = there ? row / a.G : 0, gq = there ? row - tok * a.G : 0;
        // rows of a warp's 32, two (D = 128) or four at a time: 16 bytes of a row per lane
        constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
        const int sub = lane / kLanes, ch = lane % kLanes;
        unsigned char* mine = sq + t * L::kQBytes + (ch >> 3) * 16384;
        const int64_t head = (int64_t)h * a.G * D + 8 * ch;
        // (rolled loops here and at the end: code that a block runs once is fetched cold)
        const uint32_t qdst = smem_u32(mine);
#pragma unroll 1
        for (int i = 0; i < 32; i += kAtOnce) {
            const int from = i + sub, ft = __shfl_sync(~0u, tok, from), fg = __shfl_sync(~0u, gq, from);
            const uint32_t n = row0 + t * 128 + (warp & 3) * 32 + from < rows ? 16u : 0u;   // (0: zero)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                         ::"r"(qdst + sw128((warp & 3) * 32 + from, ch & 7)),
                         "l"(a.Q + (int64_t)(s.q0 + ft) * a.ldQ + head + (int64_t)fg * D), "r"(n)
                         : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->q_full);
        const int limit = (there ? s.start + tok : -1) - ja * kTcTokens;
        const int least = s.start + (row0 + t * 128) / a.G - ja * kTcTokens;   // the tile's first row sees least
        // Weights are 2^(x - base).  base is a maximum less 8, rounded up, and moves when a score has passed it by
        // 14, rounded down, so that x - base is exact near the maximum and no weight is above 2^14.  For ordinary
        // scores -base is folded into the product's addend, which rounds by half a step of base; from kTcApart on
        // (before that takes weights out of fp16) it is subtracted on its own, in a pass of its own over the scores
        // (always: 192.4 us for the prompt of 4096, this 188.3, without it 187.0).
        float base = -INFINITY, l = 0.f;
        bool apart = false;                              // of a warp
        for (int j = 0; j < nt[t]; ++j) {
            if (ok) ok = mbar_wait(&sh->s_full[t], j & 1, a.status);
            tc_fence_after();
            const KvTcMeta& mt = sh->meta[j % kTcMeta];
            // tokens of each page that this row sees
            const int see[2] = {min(mt.valid[0], limit - j * kTcTokens + 1), min(mt.valid[1], limit - j * kTcTokens - kKvPage + 1)};
            const bool masked = row0 + t * 128 + 128 > rows || least < j * kTcTokens + kTcTokens - 1 ||
                                mt.valid[0] < kKvPage || mt.valid[1] < kKvPage;
            // a page of which the row sees nothing: any finite scale (its own may be NaN)
            float sa[2] = {see[0] > 0 ? mt.a[0] : 1.f, see[1] > 0 ? mt.a[1] : 1.f};
            const float slv[2] = {see[0] > 0 ? mt.lv[0] : 0.f, see[1] > 0 ? mt.lv[1] : 0.f};
            // 64 scores of page q (compact code: the loops over pages stay rolled)
            auto scores = [&](int q, uint32_t (&v)[64]) {
                tmem_ld64(ts + q * 64, v);
                if (masked) {                            // (the scales are above zero: -inf stays)
                    const int n = q == 0 ? see[0] : see[1];
#pragma unroll
                    for (int i = 0; i < 64; ++i) v[i] = i < n ? v[i] : 0xff800000u;
                }
            };
            float cand = see[0] > 0 || see[1] > 0 ? kLeastScore : -INFINITY;   // (a row that sees something has a maximum)
#pragma unroll 1
            for (int q = 0; q < 2; ++q) {
                uint32_t v[64];
                scores(q, v);
                float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    m[i & 3] = max3(m[i & 3], __uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
                cand = fmaxf(cand, fmaf(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), q == 0 ? sa[0] : sa[1], q == 0 ? slv[0] : slv[1]));
            }
            const bool move = cand > __fadd_rd(base, kTcWeightExp + kTcSlack);
            if (__any_sync(~0u, move)) {
                const float next = move ? __fadd_ru(cand, -kTcWeightExp) : base;   // (no row depends on its neighbours)
                if (j > 0) {
                    const float f = base == next ? 1.f : tc_ex2(base - next);
                    if (ok) ok = mbar_wait(&sh->o_done[t], (j - 1) & 1, a.status);
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t v[32];
                        tmem_ld32(to + c * 32, v);
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
                        tmem_st32(to + c * 32, v);
                    }
                    l *= f;
                }
                base = next;
                apart = __any_sync(~0u, fabsf(base) >= kTcApart && base > -INFINITY);
            }
            // a weight is 2^(a score + off)
            const float less = base == -INFINITY ? 0.f : base;
            float off[2] = {slv[0] - less, slv[1] - less};
            if (apart) {
                // here first the scores become x - base, and then the weights are of them as they are; a row whose
                // own scores are ordinary gets the same bits as without such neighbours
                const bool mine = fabsf(less) >= kTcApart;
                const float then = mine ? less : 0.f;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    const float a1 = c < 2 ? sa[0] : sa[1], add = c < 2 ? (mine ? slv[0] : off[0]) : (mine ? slv[1] : off[1]);
                    uint32_t v[32];
                    tmem_ld32(ts + c * 32, v);
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(fmaf(__uint_as_float(v[i]), a1, add) - then);
                    tmem_st32(ts + c * 32, v);
                }
                sa[0] = sa[1] = 1.f;
                off[0] = off[1] = 0.f;
            }
#pragma unroll 1
            for (int q = 0; q < 2; ++q) {
                uint32_t v[64];
                scores(q, v);
                const float aq = q == 0 ? sa[0] : sa[1], oq = q == 0 ? off[0] : off[1];
                const uint64_t a2 = pack_f2(aq, aq), o2 = pack_f2(oq, oq);
                uint64_t s2 = 0ull, s3 = 0ull;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t p[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint64_t e2 = fma_f2(pack_f2(__uint_as_float(v[c * 32 + 2 * i]), __uint_as_float(v[c * 32 + 2 * i + 1])), a2, o2);
                        float w0, w1;
                        unpack_f2(e2, w0, w1);
                        w0 = tc_ex2(w0);
                        w1 = tc_ex2(w1);
                        if (i & 1) s3 = add_f2(s3, pack_f2(w0, w1));
                        else s2 = add_f2(s2, pack_f2(w0, w1));
                        p[i] = h2_as_u32(__floats2half2_rn(w0, w1));
                    }
                    tmem_st16(ts + q * 32 + c * 16, p);  // columns whose scores this page or the one before has read
                }
                float s0, s1;
                unpack_f2(add_f2(s2, s3), s0, s1);
                const float sum = s0 + s1;
                // a row that sees nothing of a page takes nothing from its scale (which may be NaN)
                if ((q == 0 ? see[0] : see[1]) > 0) l += sum * mt.inv[q];
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->p_full[t]);
        }
        if (nt[t] > 0) {
            if (ok) ok = mbar_wait(&sh->o_done[t], (nt[t] - 1) & 1, a.status);
            tc_fence_after();
        }
        // With several shares, each leaves its O, m and l in the workspace (a column's
        // rows side by side), and the last to count joins them, in the shares' order.
        bool last = true;
        const int mrow = t * 128 + r;
        // (row tiles of the batch: no more than T G / 256 + n, however uneven the sequences)
        const int64_t tiles_before = (int64_t)s.q0 * a.G / kTcRows + b;
        float* parts = a.partial + ((tiles_before + tile) * a.c.kv_heads + h) * a.S * (D + 2) * kTcRows + mrow;
        auto column = [&](int c, uint32_t (&v)[32]) {                // O's columns from 32 c: zero where nothing was seen
            if (nt[t] > 0) {
                tmem_ld32(to + c * 32, v);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = 0u;
            }
        };
        if (shares > 1) {
            float* part = parts + (int64_t)share * (D + 2) * kTcRows;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t v[32];
                column(c, v);
#pragma unroll
                for (int i = 0; i < 32; ++i) __stcg(part + (c * 32 + i) * kTcRows, __uint_as_float(v[i]));
            }
            __stcg(part + D * kTcRows, base);
            __stcg(part + (D + 1) * kTcRows, l);
            __threadfence();
            named_barrier_sync(2, 256);
            if (threadIdx.x == 0) {
                unsigned int prev;
                asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(prev) : "l"(a.tickets + unit) : "memory");
                sh->last = prev == (unsigned)(shares - 1);
                if (sh->last) atomicExch(a.tickets + unit, 0u);      // every share has counted: ready for the next call
            }
            named_barrier_sync(2, 256);
            last = sh->last;
            __threadfence();
            if (last) {
                base = -INFINITY;
                for (int k = 0; k < shares; ++k) base = fmaxf(base, __ldcg(parts + ((int64_t)k * (D + 2) + D) * kTcRows));
                const float ref = base == -INFINITY ? 0.f : base;
                l = 0.f;
                for (int k = 0; k < shares; ++k) {
                    const float* p = parts + ((int64_t)k * (D + 2) + D) * kTcRows;
                    l = fmaf(tc_ex2(__ldcg(p) - ref), __ldcg(p + kTcRows), l);
                }
            }
        }
        if (last) {
            const float ref = base == -INFINITY ? 0.f : base;
            if (l == 0.f && base > -INFINITY) l = __int_as_float(0x7fffffff);   // every score is -inf
            const float inv = l == 0.f ? 0.f : 1.f / l;                  // a row that sees nothing is zero
            // (the tile's products are complete, so its queries' buffer takes the outputs; a warp's rows are its own)
            unsigned char* out = sq + t * L::kQBytes;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t v[32];
                if (shares == 1) {
                    column(c, v);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = 0u;
#pragma unroll 1
                    for (int k = 0; k < shares; ++k) {
                        const float* p = parts + (int64_t)k * (D + 2) * kTcRows;
                        const float f = tc_ex2(__ldcg(p + D * kTcRows) - ref);
                        uint32_t u[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(__ldcg(p + (c * 32 + i) * kTcRows));
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(fmaf(f, __uint_as_float(u[i]), __uint_as_float(v[i])));
                    }
                }
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                    uint4 y = make_uint4(0, 0, 0, 0);
                    if (l != 0.f) {
                        y.x = h2_as_u32(__floats2half2_rn(__uint_as_float(v[i]) * inv, __uint_as_float(v[i + 1]) * inv));
                        y.y = h2_as_u32(__floats2half2_rn(__uint_as_float(v[i + 2]) * inv, __uint_as_float(v[i + 3]) * inv));
                        y.z = h2_as_u32(__floats2half2_rn(__uint_as_float(v[i + 4]) * inv, __uint_as_float(v[i + 5]) * inv));
                        y.w = h2_as_u32(__floats2half2_rn(__uint_as_float(v[i + 6]) * inv, __uint_as_float(v[i + 7]) * inv));
                    }
                    const int x = c * 4 + (i >> 3);
                    *reinterpret_cast<uint4*>(out + (x >> 3) * 16384 + sw128(r, x & 7)) = y;
                }
            }
            __syncwarp();
#pragma unroll 1
            for (int i = 0; i < 32; i += 4 * kAtOnce) {
                uint4 y[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    y[k] = *reinterpret_cast<const uint4*>(mine + sw128((warp & 3) * 32 + i + k * kAtOnce + sub, ch & 7));
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int from = i + k * kAtOnce + sub, ft = __shfl_sync(~0u, tok, from), fg = __shfl_sync(~0u, gq, from);
                    if (row0 + t * 128 + (warp & 3) * 32 + from < rows)
                        *reinterpret_cast<uint4*>(a.Y + (int64_t)(s.q0 + ft) * a.ldY + head + (int64_t)fg * D) = y[k];
                }
            }
        }
    } else if (warp < 12) {
        // ---------------- pages to operands (128 threads) ----------------
        const int tid = threadIdx.x - 256;
        const int full = s.len / kKvPage - 2 * ja, ntok = s.len % kKvPage;
        const int64_t tail = ((int64_t)s.slot * a.c.kv_heads + h) * kKvPage * D;
        const int* table = a.b.table + (int64_t)b * a.b.max_pages + 2 * ja;
        constexpr int kPieces = kKvPage * D / 16 / 128;              // 16-byte pieces of a page's K (or V) per thread
        // the table's entry for page p (loaded a tile ahead of its use), and what it
        // says: the page's id, -1 absent (or out of range), -2 the tail
        auto entry = [&](int p) { return p < full && p < 2 * nmax ? ldcg_s32(table + p) : -1; };
        auto page_of = [&](int p, int id) -> int {
            if (p < full) {
                if (id >= 0 && id < a.c.pages) return id;
                if (tid == 0 && p < 2 * nmax) record_status(a.status, GLOWQ_ERR_INDEX);
                return -1;
            }
            return p == full && ntok > 0 ? -2 : -1;
        };
        // 16 codes -> 32 bytes of a swizzled row; a thread's pieces of a page are 32
        // rows apart, 4 KB in the layout, with the same chunks
        const uint32_t out0 = sw128(tid >> 2, 2 * (tid & 3)), out1 = sw128(tid >> 2, 2 * (tid & 3) + 1);
        auto codes_to = [&](const uint4& u, unsigned char* at) {
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
            uint32_t o[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) tc_cvt_codes(w[i], o[2 * i], o[2 * i + 1]);
            *reinterpret_cast<uint4*>(at + out0) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(at + out1) = make_uint4(o[4], o[5], o[6], o[7]);
        };
        // the codes of a tile's K (which = 0) or V, staged ahead by bulk copies of one thread
        auto stage_codes = [&](int which, const int (&id)[2]) {
            if (tid != 0) return;
            mbar_arrive_expect_tx(&sh->codes[which], (uint32_t)(((id[0] >= 0) + (id[1] >= 0)) * kKvPage * D));
#pragma unroll
            for (int q = 0; q < 2; ++q)
                if (id[q] >= 0)
                    bulk_g2s(smem_u32(sc + which * L::kCodes + q * kKvPage * D),
                             (which ? a.c.v_codes : a.c.k_codes) + ((int64_t)id[q] * a.c.kv_heads + h) * kKvPage * D,
                             kKvPage * D, &sh->codes[which]);
        };
        // this thread's pieces of the tail (8 dimensions of a token each), all loads in
        // flight; tokens past the end are zero
        constexpr int kTail = kKvPage * D / 8 / 128;
        auto tail_pieces = [&](const uint16_t* src, uint4 (&u)[kTail]) {
#pragma unroll
            for (int i = 0; i < kTail; ++i) {
                const int x = tid + i * 128, tok = x / (D / 8), c = x % (D / 8);
                u[i] = ldcg_128_if(src + tail + (int64_t)tok * D + 8 * c, tok < ntok);
            }
        };
        const int first[2] = {entry(0), entry(1)};
        int ahead[2] = {entry(2), entry(3)};             // the next tile's entries
        int id[2] = {page_of(0, first[0]), page_of(1, first[1])};
        float ks = 0.f, vs = 1.f;                        // thread q < 2: the scales of page q
        auto scales_of = [&](const int (&id)[2], float& k, float& v) {
            k = 0.f;
            v = 1.f;
            if (tid < 2 && id[tid] >= 0) {
                k = ldcg_f32(a.c.k_scales + (int64_t)id[tid] * a.c.kv_heads + h);
                v = ldcg_f32(a.c.v_scales + (int64_t)id[tid] * a.c.kv_heads + h);
            }
        };
        if (nmax > 0) {
            stage_codes(0, id);
            stage_codes(1, id);
            scales_of(id, ks, vs);
        }
        for (int j = 0; j < nmax; ++j) {
            const int st = j & 1;
            // the next tile's pages and scales, loaded ahead
            int nid[2] = {-1, -1};
            float nks = 0.f, nvs = 1.f;
            if (j + 1 < nmax) {
                nid[0] = page_of(2 * j + 2, ahead[0]);
                nid[1] = page_of(2 * j + 3, ahead[1]);
                scales_of(nid, nks, nvs);
                ahead[0] = entry(2 * j + 4);
                ahead[1] = entry(2 * j + 5);
            }
            KvTcMeta& mt = sh->meta[j % kTcMeta];
            if (tid < 2) {
                const int p = id[tid];
                mt.a[tid] = p == -2 ? a.scale_log2 : ks * a.scale_log2;
                mt.lv[tid] = log2f(vs);
                mt.inv[tid] = 1.f / vs;
                mt.valid[tid] = p >= 0 ? kKvPage : p == -2 ? ntok : 0;
            }
            __half2 up = __half2half2(__ushort_as_half(0x3c00));     // the tail's power of two (attention.cu)
            if (id[0] == -2 || id[1] == -2) {
                const int q = id[0] == -2 ? 0 : 1;
                if (tid == 0) sh->tail_max = sh->tail_poison[0] = sh->tail_poison[1] = 0u;
                named_barrier_sync(1, 128);
                __half2 am = __half2half2(__ushort_as_half(0));
                uint4 tv[kTail];
                tail_pieces(a.c.v_tail, tv);
#pragma unroll
                for (int n = 0; n < kTail; ++n) {
                    const int i = tid + n * 128;
                    const uint32_t w[4] = {tv[n].x, tv[n].y, tv[n].z, tv[n].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t x = w[e];
                        const bool lo = (x & 0x7c00u) == 0x7c00u, hi = (x & 0x7c000000u) == 0x7c000000u;
                        if (lo) x &= 0xffff0000u;
                        if (hi) x &= 0x0000ffffu;
                        if (lo || hi) atomicOr(&sh->tail_poison[i / (D / 8) >> 5], 1u << (i / (D / 8) & 31));
                        am = __hmax2(am, __habs2(u32_as_h2(x)));
                    }
                }
                atomicMax(&sh->tail_max, max(h2_as_u32(am) & 0x7c00u, (h2_as_u32(am) >> 16) & 0x7c00u) >> 10);
                named_barrier_sync(1, 128);
                const int k2 = min(15, 21 - (int)sh->tail_max);
                up = __half2half2(__ushort_as_half((unsigned short)((k2 + 15) << 10)));
                if (tid == 0) {
                    mt.lv[q] = (float)-k2;
                    mt.inv[q] = exp2f((float)k2);
                }
            }
            // The complete pages of a tile's K (which = 0) or V, from the staged codes.
            // One rolled body for both: a thread's pieces i of a page are rows 32 apart
            // (4 KB), and of K's second panel 16 KB, of V's second 64 dimensions 8 KB on.
            auto convert = [&](int which, unsigned char* to, int half, int page) {
                if (ok) ok = mbar_wait(&sh->codes[which], j & 1, a.status);
                const unsigned char* from = sc + which * L::kCodes + tid * 16;
#pragma unroll 1
                for (int q = 0; q < 2; ++q, from += kKvPage * D, to += page) {
                    if ((q ? id[1] : id[0]) < 0) continue;
                    uint4 u[kPieces];
#pragma unroll
                    for (int i = 0; i < kPieces; ++i) u[i] = *reinterpret_cast<const uint4*>(from + i * 2048);
#pragma unroll
                    for (int i = 0; i < kPieces; ++i) codes_to(u[i], to + (i & 1) * 4096 + (i >> 1) * half);
                }
            };
            // The codes' buffer may be filled again only behind the conversion, which
            // has waited for the reads: a barrier behind the reads alone lets a bulk
            // copy overtake them (seen at D = 64: a tile read its successor's values).
            auto next_codes = [&](int which) {
                if (j + 1 < nmax) {
                    fence_proxy_async_smem();
                    named_barrier_sync(1, 128);
                    stage_codes(which, nid);
                }
            };
            // ---- K ----
            if (j >= 2 && ok) ok = mbar_wait(&sh->ke[st], ((j >> 1) - 1) & 1, a.status);
            unsigned char* kd = sk + st * L::kKBytes;
            convert(0, kd, 16384, 8192);
            if (id[0] < 0 || id[1] < 0) {
#pragma unroll 1
                for (int q = 0; q < 2; ++q) {
                    const int p = q ? id[1] : id[0];
                    if (p >= 0) continue;
                    uint4 tk[kTail];
#pragma unroll
                    for (int n = 0; n < kTail; ++n) tk[n] = make_uint4(0, 0, 0, 0);
                    if (p == -2) tail_pieces(a.c.k_tail, tk);
#pragma unroll
                    for (int n = 0; n < kTail; ++n) {
                        const int i = tid + n * 128, tok = i / (D / 8), c = i % (D / 8);
                        // a token whose value is not finite (taken out of V): scores NaN for the rows that see it
                        if (p == -2 && ((sh->tail_poison[tok >> 5] >> (tok & 31)) & 1u)) tk[n] = make_uint4(~0u, ~0u, ~0u, ~0u);
                        *reinterpret_cast<uint4*>(kd + (c >> 3) * 16384 + sw128(q * kKvPage + tok, c & 7)) = tk[n];
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->kf[st]);
            next_codes(0);
            // ---- V ----
            if (j >= 2 && ok) ok = mbar_wait(&sh->ve[st], ((j >> 1) - 1) & 1, a.status);
            unsigned char* vd = sv + st * L::kVBytes;
            convert(1, vd, 8192, D * 128);
            if (id[0] < 0 || id[1] < 0) {
#pragma unroll 1
                for (int q = 0; q < 2; ++q) {
                    const int p = q ? id[1] : id[0];
                    unsigned char* page = vd + q * D * 128;
                    if (p == -2) {
                        uint4 tv[kTail];
                        tail_pieces(a.c.v_tail, tv);
#pragma unroll
                        for (int n = 0; n < kTail; ++n) {
                            const int i = tid + n * 128, tok = i / (D / 8), dim = i % (D / 8) * 8;
                            uint32_t w[4] = {tv[n].x, tv[n].y, tv[n].z, tv[n].w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if ((w[e] & 0x7c00u) == 0x7c00u) w[e] &= 0xffff0000u;
                                if ((w[e] & 0x7c000000u) == 0x7c000000u) w[e] &= 0x0000ffffu;
                                const __half2 x = __hmul2(u32_as_h2(w[e]), up);
                                *reinterpret_cast<__half*>(page + sw128(dim + 2 * e, tok >> 3) + (tok & 7) * 2) = __low2half(x);
                                *reinterpret_cast<__half*>(page + sw128(dim + 2 * e + 1, tok >> 3) + (tok & 7) * 2) = __high2half(x);
                            }
                        }
                    } else if (p == -1) {
                        for (int i = tid; i < D * 8; i += 128) *reinterpret_cast<uint4*>(page + i * 16) = make_uint4(0, 0, 0, 0);
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->vf[st]);
            next_codes(1);
            id[0] = nid[0];
            id[1] = nid[1];
            ks = nks;
            vs = nvs;
        }
    } else if (warp == 12 && nmax > 0) {
        // ---------------- MMA issuer (the whole warp; one lane issues) ----------------
        const uint32_t ids = f16_idesc(128, kTcTokens), ido = f16_idesc(128, D);
        const uint64_t qd = sw128_kmajor_desc(smem_u32(sq)), kd = sw128_kmajor_desc(smem_u32(sk)), vd = sw128_kmajor_desc(smem_u32(sv));
        auto qk = [&](int t, int st) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {                       // panels of 64 dimensions 16 KB apart
                const uint64_t off = (uint64_t)((k >> 2) * 1024 + (k & 3) * 2);
                umma_ss_elect(tmem + (uint32_t)(t * 128), qd + (uint64_t)(t * (L::kQBytes >> 4)) + off,
                              kd + (uint64_t)(st * (L::kKBytes >> 4)) + off, ids, k > 0);
            }
            umma_commit_elect(smem_u32(&sh->s_full[t]));
        };
        ok = mbar_wait_warp(smem_u32(&sh->q_full), 0, a.status);
        if (ok) ok = mbar_wait_warp(smem_u32(&sh->kf[0]), 0, a.status);
        tc_fence_after();
        for (int t = 0; t < 2; ++t)
            if (nt[t] > 0) qk(t, 0);
        umma_commit_elect(smem_u32(&sh->ke[0]));
        for (int j = 0; j < nmax; ++j) {
            const int st = j & 1, sn = st ^ 1;
            if (ok) ok = mbar_wait_warp(smem_u32(&sh->vf[st]), (j >> 1) & 1, a.status);
            if (j + 1 < nmax && ok) ok = mbar_wait_warp(smem_u32(&sh->kf[sn]), ((j + 1) >> 1) & 1, a.status);
            for (int t = 0; t < 2; ++t) {
                if (j >= nt[t]) continue;
                if (ok) ok = mbar_wait_warp(smem_u32(&sh->p_full[t]), j & 1, a.status);
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < kTcTokens / 16; ++k)             // pages of 64 tokens D rows apart
                    umma_ts_elect(tmem + (uint32_t)(256 + t * 128), tmem + (uint32_t)(t * 128 + k * 8),
                                  vd + (uint64_t)(st * (L::kVBytes >> 4) + (k >> 2) * (D * 8) + (k & 3) * 2), ido, j > 0 || k > 0);
                umma_commit_elect(smem_u32(&sh->o_done[t]));
                if (j + 1 < nt[t]) qk(t, sn);
            }
            umma_commit_elect(smem_u32(&sh->ve[st]));
            if (j + 1 < nmax) umma_commit_elect(smem_u32(&sh->ke[sn]));
        }
        // the last commits land before the block may exit
        for (int j = (nmax > 2 ? nmax - 2 : 0); j < nmax; ++j) {
            if (ok) ok = mbar_wait_warp(smem_u32(&sh->ke[j & 1]), (j >> 1) & 1, a.status);
            if (ok) ok = mbar_wait_warp(smem_u32(&sh->ve[j & 1]), (j >> 1) & 1, a.status);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 12) tmem_dealloc(tmem, 512);
}

template <int D>
static cudaError_t launch_tc(const KvTcArgs& a, unsigned grid, cudaStream_t st) {
    static SmemLimit limit;
    cudaError_t e = limit.raise((const void*)kv_attention_tc_kernel<D>, KvTc<D>::kSmem);
    if (e != cudaSuccess) return e;
    void* args[] = {(void*)&a};
    return launch_pdl((const void*)kv_attention_tc_kernel<D>, grid, kTcThreads, KvTc<D>::kSmem, st, args);
}

// Shares of a unit's tokens: what their number is expected to take, the tables
// being full, is 2.7 us for a tile of 128 tokens and 6.4 us for the rest of a block,
// in waves of a block for each SM; with shares 8 us more of a block and 2 us for
// each part of the join.  (512 rows of one sequence and 8 kv heads after 32768
// tokens: 635 us whole, 112 us in nine shares; of eight sequences after 2048
// tokens, where each SM has a block: 61 us whole, 87 us in three.)
KvTcShares kv_tc_shares(const KvBatchView& b, int G, int kv_heads, int num_sms) {
    const int64_t rt = ((int64_t)b.max_new * G + kTcRows - 1) / kTcRows, grid = rt * b.n_seq * kv_heads;
    // units: no more than T G / 256 + n row tiles, however uneven the sequences
    const int64_t all = ((int64_t)b.T * G / kTcRows + b.n_seq) * kv_heads, units = grid < all ? grid : all;
    const double tiles = ((int64_t)b.max_pages * kKvPage + kTcTokens - 1) / kTcTokens;
    KvTcShares best = {1, 0.};
    for (int S = 1; S <= kTcMostShares; ++S) {
        if (S > 1 && (tiles < (double)S * kTcLeastTiles || grid > kTcMostTickets)) break;
        const double waves = (double)((units * S + num_sms - 1) / num_sms);
        const double us = waves * (tiles / S * 2.7 + 6.4 + (S > 1 ? 8. : 0.)) + (S > 1 ? 2. * S : 0.);
        if (S == 1 || us < best.us) best = {S, us};
    }
    return best;
}
size_t kv_tc_partial_bytes(const KvBatchView& b, int G, int kv_heads, int S, int head_dim) {
    const int64_t tiles = (int64_t)b.T * G / kTcRows + b.n_seq;
    return S > 1 ? (size_t)tiles * kv_heads * S * (head_dim + 2) * kTcRows * sizeof(float) : 0;
}
cudaError_t launch_kv_attention_tc(const KvCacheView& c, const KvBatchView& b, const uint16_t* Q, int64_t ldQ, int q_heads,
                                   float scale, uint16_t* Y, int64_t ldY, unsigned int* tickets, float* partial, int S,
                                   cudaStream_t st) {
    const int G = q_heads / c.kv_heads;
    // above zero, so that a masked score of -inf stays one (below 1e-25 every score is zero beside fp32's steps)
    const float scale_log2 = scale > 1e-25f ? scale * 1.44269504088896340736f : 1e-25f;
    const KvTcArgs a = {c, b, Q, Y, ldQ, ldY, scale_log2, G,
                        (int)(((int64_t)b.max_new * G + kTcRows - 1) / kTcRows), S, partial, tickets, device_status_ptr()};
    const unsigned grid = (unsigned)((int64_t)a.rt * b.n_seq * c.kv_heads * S);
    return c.head_dim == 64 ? launch_tc<64>(a, grid, st) : launch_tc<128>(a, grid, st);
}

}  // namespace glowq
