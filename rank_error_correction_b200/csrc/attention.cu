// attention.cu -- causal attention of a step's queries over the paged 8-bit
// key/value cache.
//
//   o_i = sum_j softmax_j(scale q_i . k_j) v_j,   j <= len - n + i  (n new rows)
//
// Products of a complete page are integer products: its codes as they are, the
// queries as 24-bit fixed point numbers in three 8-bit digits (exact but for
// elements below 2^-11 of their row's largest, which are off by 2^-23 of it at
// most), the weights as 24-bit ones of the page's largest in their row (off by
// 2^-24 of it).  Digits' sums are exact in 32 bits and joined in fp32.  (Codes
// turned into fp16 for fp16 products took as long, 109 us against 111 at 100,000
// tokens when both were measured, and round every weight to 2^-11.)  The page's scales meet the sums in fp32, s_K on the
// scores, and s_V inside the exponent, as
//   w_ij = 2^(x_ij + log2 s_V - m_i),  x_ij = scale log2(e) s_K q_i . k_j
// with m_i the running maximum of x + log2 s_V.  The numerator is then
// sum_j w_ij v_j with integer v, and the denominator sum_pages (sum_j w_ij) / s_V.
// An incomplete last page is fp16, and its products are: weights, scaled by 2^8
// (the factor cancels; fp16's smallest normal is then 2^-22 of the largest), are
// the sum of two fp16 numbers (off by 2^-24 of themselves and 2^-33 of the
// largest).  Sums, maxima and outputs in fp32.
#include <climits>

#include "common.cuh"
#include "internal.cuh"
#include "kvcache.cuh"
#include "quant8.cuh"

namespace glowq {

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = kAttnWarps * 32;
constexpr int kAttnRing = 4;             // chunks of 4 KB of a warp's ring
constexpr int kAttnParts = 128;          // blocks that share one unit, at most (and the two at its ends)
constexpr int kAttnUnitCost = 10;        // what a unit costs beyond its pages, in pages
constexpr int kAttnLeastShare = kAttnUnitCost + 2 * kAttnWarps;
constexpr float kWeightExp = 8.f;

struct KvAttnArgs {
    KvCacheView c;
    KvBatchView b;
    const uint16_t* Q;
    uint16_t* Y;
    int64_t ldQ, ldY;
    float scale_log2;        // scale log2(e)
    int G, sms;
    float* partial;          // [block][2][8 RN][D + 4]
    unsigned int* tickets;   // [block], zero between calls
    unsigned int* status;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ uint32_t movm(uint32_t x) {            // 8 x 8 fp16 matrix across the warp, transposed
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void mma_s8(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, const int (&c)[4]) {
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "r"(c[0]), "r"(c[1]), "r"(c[2]), "r"(c[3]));
}
__device__ __forceinline__ void mma_s8u8(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, const int (&c)[4]) {
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.u8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "r"(c[0]), "r"(c[1]), "r"(c[2]), "r"(c[3]));
}
// Digits' sums as fp32.  A sum starts from the bits of 1.5 2^23, so that its bits
// are the float 1.5 2^23 + sum (|sum| <= 128 * 128 * 128 < 2^22); two of them:
// 2^16 hi + 2^8 mid + lo, the first step exact.
constexpr int kSumBits = 0x4b400000;
__device__ __forceinline__ uint64_t join_f2(const int* hi, const int* mid, const int* lo) {
    const float b = 12582912.f, c = -12582912.f * 65792.f;
    const uint64_t h = pack_f2(__int_as_float(hi[0]), __int_as_float(hi[1])), m = pack_f2(__int_as_float(mid[0]), __int_as_float(mid[1]));
    const uint64_t l = add_f2(pack_f2(__int_as_float(lo[0]), __int_as_float(lo[1])), pack_f2(-b, -b));
    return add_f2(fma_f2(m, pack_f2(256.f, 256.f), fma_f2(h, pack_f2(65536.f, 65536.f), pack_f2(c, c))), l);
}
// Returns when this warp's loads behind x have arrived: what they read may be overwritten.
__device__ __forceinline__ void arrived(uint32_t x) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.eq.u32 p, %0, 1;\n\tvote.sync.any.pred q, p, 0xffffffff;\n\t}" ::"r"(x)
        : "memory");
}

// Running softmax of a warp's 8 RN rows.  Scores come as S^T = K Q^T and outputs
// as O^T = V^T P^T: with the tokens in the MMA's rows, as few as 8 query rows
// fill its columns (16 in its rows would be half empty for most decode steps:
// the products took twice the instructions and the softmax twice the registers).
// This lane: query rows 8 r + 2 t + e; tokens (dimensions) g and g + 8 of a tile.
template <int D, int RN>
struct AttnState {
    float m[RN][2], l[RN][2], o[RN][D / 16][4];          // l: this lane's tokens only
};

// One tile of 16 tokens of a tail, at column g and g + 8 in this lane; lim: last
// visible token of each query row; lv = log2 of the tail's unit.  Returns the
// weights as B fragments (k = tokens, n = query rows), each in two fp16 terms:
// what the first is off by (2^-12 of the weight), to another 2^-12.
template <int D, int RN>
__device__ __forceinline__ void softmax_tail(AttnState<D, RN>& st, float (&x)[RN][4], const int (&lim)[RN][2], float xs, float lv,
                                             float inv_sv, int g, uint32_t (&pf)[RN][2][2]) {
    float corr[RN][2];
    bool moved = false;
#pragma unroll
    for (int r = 0; r < RN; ++r) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[r][e] = g + 8 * (e >> 1) > lim[r][e & 1] ? -INFINITY : fmaf(x[r][e], xs, lv);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float m = fmaxf(x[r][e], x[r][e + 2]);
            m = fmaxf(m, __shfl_xor_sync(~0u, m, 4));
            m = fmaxf(m, __shfl_xor_sync(~0u, m, 8));
            m = fmaxf(st.m[r][e], fmaxf(m, __shfl_xor_sync(~0u, m, 16)));
            const float ref = m == -INFINITY ? 0.f : m;               // nothing visible yet: weights 2^-inf = 0
            corr[r][e] = ex2(st.m[r][e] - ref);
            moved |= corr[r][e] != 1.f;
            st.m[r][e] = m;
            x[r][e] = ex2(x[r][e] - ref + kWeightExp);               // (x - ref is exact where it matters, however large they are)
            x[r][e + 2] = ex2(x[r][e + 2] - ref + kWeightExp);
            st.l[r][e] = fmaf(x[r][e] + x[r][e + 2], inv_sv, st.l[r][e] * corr[r][e]);
        }
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            const __half2 h = __floats2half2_rn(x[r][e], x[r][e + 1]);
            const float2 f = __half22float2(h);
            pf[r][0][e >> 1] = movm(h2_as_u32(h));
            pf[r][1][e >> 1] = movm(h2_as_u32(__floats2half2_rn(x[r][e] - f.x, x[r][e + 1] - f.y)));
        }
    }
    if (__any_sync(~0u, moved)) {
#pragma unroll
        for (int r = 0; r < RN; ++r)
#pragma unroll
            for (int n = 0; n < D / 16; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) st.o[r][n][e] *= corr[r][e & 1];
    }
}

// Units of work: 8 RN query rows (row = new token i and query head gq of the kv
// head's group, i G + gq) of one sequence and kv head, a page at a time.
struct AttnSpan {
    int pages, tiles;                                    // of a sequence: pages (1 at least), tiles of rows
    __device__ long long all(int heads) const { return (long long)(pages + kAttnUnitCost) * tiles * heads; }
};
template <int RN>
__device__ __forceinline__ AttnSpan attn_span(const KvSeq& s, const KvBatchView& b, int G) {
    const int p = s.len <= (int64_t)b.max_pages * kKvPage ? (s.len + kKvPage - 1) / kKvPage : 1;
    return {max(p, 1), (int)(((int64_t)s.nq * G + 8 * RN - 1) / (8 * RN))};
}

// The pages of all units, in a row, are cut into equal shares, one for each
// block: sequences of any lengths keep every SM busy to the end (a block for
// each sequence and head left half of the GPU idle behind the longest).  A unit
// starts with kAttnUnitCost empty pages, for its queries, its tail and its results
// (without them the shares of the shortest sequences, ten units each, took twice
// as long as the others).  A block takes its share unit by unit; its warps take the pages in turn, each with a
// ring of K and V half-pages filled by bulk copies; lane (g, t) feeds the MMA 16
// consecutive bytes of a row at a time (k in the order 16 t + 4 step, the same in
// both operands).  The tokens of an incomplete last page are split among the
// warps.  The warps' results meet in shared memory, the shares' in the
// workspace: the block that counts last on a unit adds its parts in order.
// Bound by memory where there is enough of it: two sequences of 116,000 and
// 126,000 tokens, 8 kv heads of 128: 497 MB in 92 us, 82 % of the copy bandwidth;
// 64 sequences of 1 to 4096 tokens: 252 MB in 61 us, 64 % (each of 2.2 units of a
// block drains its ring, and pays its tail and its merge).  One sequence of 500
// tokens takes 11 us, all of it latency: lengths, page ids, codes, tail, results.
template <int D, int RN>
__global__ void __launch_bounds__(kAttnThreads, RN == 1 ? 3 : 2) kv_attention_kernel(const __grid_constant__ KvAttnArgs a) {
    constexpr int kChunk = kKvPage * 64;                 // what a bulk copy brings: 64 dimensions of a page's K or V
    constexpr int kPanels = D / 64, kRows = 8 * RN, kPart = D + 4;
    extern __shared__ __align__(128) unsigned char sm[];
    // [4 warps][ring] (later the warps' outputs, or the parts' factors), m / l of the warps
    float* sml = reinterpret_cast<float*>(sm + kAttnWarps * kAttnRing * kChunk);
    __shared__ uint64_t bars[kAttnWarps * kAttnRing];
    __shared__ long long wsum[kAttnWarps];
    __shared__ int wmax[kAttnWarps], first_seq, last_part;
    __shared__ long long first_off;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    if (tid == 0) {
        for (int i = 0; i < kAttnWarps * kAttnRing; ++i) mbar_init(bars + i, 1);
        fence_mbar_init();
    }
    pdl_wait();
    pdl_launch_dependents();
    // ---- this block's share [lo, hi) of all pages ----
    const int each = (a.b.n_seq + kAttnThreads - 1) / kAttnThreads;
    const int b0 = min(a.b.n_seq, tid * each), b1 = min(a.b.n_seq, b0 + each);
    long long mine = 0;
    int most = 0;
    for (int b = b0; b < b1; ++b) {
        const KvSeq s = kv_sequence(a.b, b);
        if (!s.ok) record_status(a.status, GLOWQ_ERR_INDEX);
        const AttnSpan w = attn_span<RN>(s, a.b, a.G);
        mine += w.all(a.c.kv_heads);
        if (w.tiles > 0) most = max(most, w.pages + kAttnUnitCost);
    }
    long long upto = mine;                               // inclusive sum over the threads
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(~0u, upto, o);
        if (lane >= o) upto += v;
        most = max(most, __shfl_xor_sync(~0u, most, o));
    }
    if (lane == 31) {
        wsum[warp] = upto;
        wmax[warp] = most;
    }
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) {
        if (w < warp) upto += wsum[w];
        total += wsum[w];
        most = max(most, wmax[w]);
    }
    // two pages for each warp at least; a unit in kAttnParts shares at most
    const long long per = max(max((total + gridDim.x - 1) / gridDim.x, (long long)kAttnLeastShare), (long long)(most + kAttnParts - 1) / kAttnParts);
    // Chunks in flight: with three blocks on an SM two of a warp's are 96 KB on the SM
    // and keep memory busy; four only queue up (100,000 tokens: 125 us against 115).
    // Fewer blocks need the four (one sequence: 14.3 us against 16.4).
    const int depth = total > 2 * a.sms * per ? 2 : kAttnRing;
    long long lo = blockIdx.x * per;
    const long long hi = min(total, lo + per);
    if (lo >= hi) return;
    if (lo >= upto - mine && lo < upto) {
        long long off = lo - (upto - mine);
        int b = b0;
        for (; b < b1; ++b) {
            const long long n = attn_span<RN>(kv_sequence(a.b, b), a.b, a.G).all(a.c.kv_heads);
            if (off < n) break;
            off -= n;
        }
        first_seq = b;
        first_off = off;
    }
    __syncthreads();
    int b = first_seq;
    long long off = first_off;                           // within the sequence's pages of all heads and tiles
    unsigned char* ring = sm + warp * kAttnRing * kChunk;
    uint64_t* wbar = bars + warp * kAttnRing;
    uint32_t phases = 0;                                 // bit i: parity of ring entry i
    bool ok = true;

    while (lo < hi) {
        const KvSeq s = kv_sequence(a.b, b);
        const AttnSpan w = attn_span<RN>(s, a.b, a.G);
        if (off >= w.all(a.c.kv_heads)) {
            off = 0;
            ++b;
            continue;
        }
        const int unit = (int)(off / (w.pages + kAttnUnitCost)), at = (int)(off - (long long)unit * (w.pages + kAttnUnitCost));
        const int h = unit % a.c.kv_heads, row0 = unit / a.c.kv_heads * kRows, rows = s.nq * a.G;
        const int take = (int)min(hi - lo, (long long)(w.pages + kAttnUnitCost - at));
        const int pa = max(0, at - kAttnUnitCost), pe = at + take - kAttnUnitCost;   // the share's pages of this unit
        if (pe <= pa) {
            lo += take;
            off += take;
            continue;
        }
        // a length that the table or the tails cannot hold: nothing is visible, and the rows are zero
        const bool tailed = s.len % kKvPage != 0;
        const bool bad = s.len > (int64_t)a.b.max_pages * kKvPage || (tailed && (s.slot < 0 || s.slot >= a.c.slots));
        if (bad && tid == 0) record_status(a.status, GLOWQ_ERR_INDEX);
        const int last_tok = min(row0 + kRows - 1, rows - 1) / a.G;  // the tile's last new token
        const int seen = bad ? 0 : max(0, s.start + last_tok + 1);   // tokens that the tile sees
        const int pb = min((seen + kKvPage - 1) / kKvPage, pe);
        const int full = s.len / kKvPage, pc = min(pb, full);        // pages in codes: [pa, pc); a tail page may follow
        const int ntok = s.len - full * kKvPage;                     // tokens of the tail
        const int64_t tail = ((int64_t)s.slot * a.c.kv_heads + h) * kKvPage * D;
        const int* table = a.b.table + (int64_t)b * a.b.max_pages;
        const bool tails = pc < pb && warp * 16 < ntok;
        if (tails) {                                                 // on its way while the pages are worked on
            constexpr int kLines = 16 * D * 2 / 128;
            if (lane < kLines && (warp * 16 + lane * 64 / D) < ntok) {
                const char* k = reinterpret_cast<const char*>(a.c.k_tail + tail + warp * 16 * D) + lane * 128;
                const char* v = reinterpret_cast<const char*>(a.c.v_tail + tail + warp * 16 * D) + lane * 128;
                asm volatile("prefetch.global.L2 [%0];\n\tprefetch.global.L2 [%1];" ::"l"(k), "l"(v));
            }
        }
        // Q's digits (lowest first) as B fragments: step q of panel p: dimensions 64 p + 16 t + 8 q .. + 7 of query
        // row 8 r + g; xq: 2^(e - 22) scale log2(e) of rows 8 r + 2 t + e, where the largest element is below 2^e
        uint32_t qd[RN][3][kPanels][4];
        float xq[RN][2];
#pragma unroll
        for (int r = 0; r < RN; ++r) {
            const int row = row0 + 8 * r + g;
            const uint16_t* q = a.Q + (int64_t)(s.q0 + row / a.G) * a.ldQ + (int64_t)(h * a.G + row % a.G) * D + 16 * t;
            uint4 u[kPanels][2];
            __half2 am = __half2half2(__ushort_as_half(0));
#pragma unroll
            for (int i = 0; i < 2 * kPanels; ++i) u[i >> 1][i & 1] = ldcg_128_if(q + 64 * (i >> 1) + 8 * (i & 1), row < rows);
#pragma unroll
            for (int i = 0; i < 2 * kPanels; ++i) amax8(u[i >> 1][i & 1], am);
            am = __hmax2_nan(am, __shfl_xor_sync(~0u, am, 1));
            am = __hmax2_nan(am, __shfl_xor_sync(~0u, am, 2));
            const float amax = amax_float(am);
            const int e = min(max((int)(__float_as_uint(amax) >> 23), 100), 143) - 126;
            const float up = __int_as_float((22 - e + 127) << 23);
            const float mine = amax <= 65504.f ? __int_as_float((e - 22 + 127) << 23) * a.scale_log2 : __int_as_float(0x7fffffff);
#pragma unroll
            for (int e2 = 0; e2 < 2; ++e2) xq[r][e2] = __shfl_sync(~0u, mine, (2 * t + e2) * 4);
#pragma unroll
            for (int i = 0; i < 4 * kPanels; ++i) {                  // four elements: two words of u
                const uint4& w4 = u[i >> 2][(i >> 1) & 1];
                const uint32_t w0 = i & 1 ? w4.z : w4.x, w1 = i & 1 ? w4.w : w4.y;
                const float2 f0 = __half22float2(u32_as_h2(w0)), f1 = __half22float2(u32_as_h2(w1));
                const float f[4] = {f0.x, f0.y, f1.x, f1.y};
                uint32_t d[3][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int v = __float_as_int(fmaf(f[j], up, 12582912.f)) - kSumBits, v1 = (v + 128) >> 8;
                    d[0][j] = v;
                    d[1][j] = v1;
                    d[2][j] = (v1 + 128) >> 8;
                }
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    qd[r][k][i >> 2][i & 3] = __byte_perm(__byte_perm(d[k][0], d[k][1], 0x0040), __byte_perm(d[k][2], d[k][3], 0x0040), 0x5410);
            }
        }
        AttnState<D, RN> st;
        int limit[RN][2];                                            // last visible position of query rows 8 r + 2 t + e
#pragma unroll
        for (int r = 0; r < RN; ++r) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = row0 + 8 * r + 2 * t + e;
                limit[r][e] = row < rows ? s.start + row / a.G : -1;
                st.m[r][e] = -INFINITY;
                st.l[r][e] = 0.f;
            }
#pragma unroll
            for (int n = 0; n < D / 16; ++n) st.o[r][n][0] = st.o[r][n][1] = st.o[r][n][2] = st.o[r][n][3] = 0.f;
        }
        const int least = row0 + kRows > rows ? -1 : s.start + row0 / a.G;   // no column behind it is masked
        int from = INT_MAX;                                          // the first position that this warp's tokens have

        // this warp's pages pa + warp, + 4, ...: page ids and scales of 32 at a time, one in each lane
        for (int p0 = pa + warp; p0 < pc; p0 += 32 * kAttnWarps) {
            const int n = min(32, (pc - p0 + kAttnWarps - 1) / kAttnWarps);
            int id = -1;
            float ks = 0.f, vs = 1.f;
            if (lane < n) {
                id = ldcg_s32(table + p0 + lane * kAttnWarps);
                if (id < 0 || id >= a.c.pages) {
                    record_status(a.status, GLOWQ_ERR_INDEX);
                    id = -1;
                } else {
                    ks = ldcg_f32(a.c.k_scales + (int64_t)id * a.c.kv_heads + h);
                    vs = ldcg_f32(a.c.v_scales + (int64_t)id * a.c.kv_heads + h);
                }
            }
            const unsigned present = __ballot_sync(~0u, id >= 0);
            if (from == INT_MAX && present) from = (p0 + (__ffs(present) - 1) * kAttnWarps) * kKvPage;
            const float lvs = log2f(vs), ivs = 1.f / vs;
            auto fetch = [&](int f) {                                // chunks in the order K, V of each page
                const int page = __shfl_sync(~0u, id, f / (2 * kPanels) & 31);
                if (f < 2 * kPanels * n && page >= 0 && lane == 0) {
                    const int c = f % (2 * kPanels);
                    const int64_t at = (((int64_t)page * a.c.kv_heads + h) * kPanels + c % kPanels) * kChunk;
                    uint64_t* bar = wbar + f % kAttnRing;
                    mbar_arrive_expect_tx(bar, kChunk);
                    bulk_g2s(smem_u32(ring + (f % kAttnRing) * kChunk), (c < kPanels ? a.c.k_codes : a.c.v_codes) + at, kChunk, bar);
                }
            };
            for (int f = 0; f < depth; ++f) fetch(f);
            for (int k = 0; k < n; ++k) {
                const int f0 = 2 * kPanels * k;
                if (__shfl_sync(~0u, id, k) < 0) {                   // not there: skipped, nothing was fetched
                    for (int f = 0; f < 2 * kPanels; ++f) fetch(f0 + f + depth);
                    continue;
                }
                const int p = p0 + k * kAttnWarps;
                const int sums0[4] = {kSumBits, kSumBits, kSumBits, kSumBits};
                const float ksc = __shfl_sync(~0u, ks, k), lv = __shfl_sync(~0u, lvs, k), iv = __shfl_sync(~0u, ivs, k);
                auto wait = [&](int f) {                             // chunk f's slot of the ring
                    const int slot = f % kAttnRing;
                    if (ok) ok = mbar_wait(wbar + slot, (phases >> slot) & 1, a.status);
                    phases ^= 1u << slot;
                    return ring + slot * kChunk;
                };
                const unsigned char* kp[kPanels];
#pragma unroll
                for (int pn = 0; pn < kPanels; ++pn) kp[pn] = wait(f0 + pn) + (16 * (g >> 1) + (g & 1)) * 64 + 16 * t;
                float x[RN][4][4];                                   // x + log2 s_V
                uint32_t seen_words = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {                        // rows g and g + 8: tokens 16 (g / 2) + 4 i + g % 2 and + 2
                    int sum[RN][3][4];
#pragma unroll
                    for (int pn = 0; pn < kPanels; ++pn) {
                        const uint4 u = *reinterpret_cast<const uint4*>(kp[pn] + 4 * i * 64);
                        const uint4 v = *reinterpret_cast<const uint4*>(kp[pn] + (4 * i + 2) * 64);
                        const uint32_t a0[4] = {u.x, v.x, u.y, v.y}, a1[4] = {u.z, v.z, u.w, v.w};
                        seen_words |= u.w | v.w;
#pragma unroll
                        for (int r = 0; r < RN; ++r)
#pragma unroll
                            for (int d = 0; d < 3; ++d) {
                                if (pn == 0) mma_s8(sum[r][d], a0, qd[r][d][pn][0], qd[r][d][pn][1], sums0);
                                else mma_s8(sum[r][d], a0, qd[r][d][pn][0], qd[r][d][pn][1], sum[r][d]);
                                mma_s8(sum[r][d], a1, qd[r][d][pn][2], qd[r][d][pn][3], sum[r][d]);
                            }
                    }
#pragma unroll
                    for (int r = 0; r < RN; ++r) {
                        const uint64_t xs = pack_f2(xq[r][0] * ksc, xq[r][1] * ksc), l2 = pack_f2(lv, lv);
#pragma unroll
                        for (int e = 0; e < 4; e += 2)
                            unpack_f2(fma_f2(join_f2(sum[r][2] + e, sum[r][1] + e, sum[r][0] + e), xs, l2), x[r][i][e], x[r][i][e + 1]);
                    }
                }
                arrived(seen_words);
#pragma unroll
                for (int pn = 0; pn < kPanels; ++pn) fetch(f0 + pn + depth);
                if (least < p * kKvPage + kKvPage - 1) {
#pragma unroll
                    for (int r = 0; r < RN; ++r)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (p * kKvPage + 16 * (g >> 1) + 4 * i + (g & 1) + 2 * (e >> 1) > limit[r][e & 1]) x[r][i][e] = -INFINITY;
                }
                // Weights 2^23 of the page's largest, and their bytes as B fragments (k = tokens, n = query rows).
                // What 2^23 stands for is base = mx - 23 rounded up, of which the joining factor `to` is made too:
                // x - base is exact near the maximum and never above 23, so that no weight passes its 24 bits
                // however large the scores are (23 - mx, rounded, did from 2^24 on: x + 23 - mx could be 24 or more).
                uint32_t pd[RN][3][4];
                float to[RN][2];                                     // what one of them weighs
                bool moved = false;
                float corr[RN][2];
#pragma unroll
                for (int r = 0; r < RN; ++r) {
                    float base[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = fmaxf(x[r][0][e], x[r][0][e + 2]);
#pragma unroll
                        for (int i = 1; i < 4; ++i) mx = max3(mx, x[r][i][e], x[r][i][e + 2]);
                        mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 16));
                        base[e] = mx == -INFINITY ? 0.f : __fadd_ru(mx, -23.f);   // (nothing visible: weights 2^-inf = 0)
                        const float m = fmaxf(st.m[r][e], mx), ref = m == -INFINITY ? 0.f : m;
                        corr[r][e] = ex2(st.m[r][e] - ref);
                        to[r][e] = mx == -INFINITY ? 0.f : ex2(base[e] - ref + kWeightExp);
                        moved |= corr[r][e] != 1.f;
                        st.m[r][e] = m;
                    }
                    const uint64_t b2 = pack_f2(-base[0], -base[1]), one = pack_f2(8388608.f, 8388608.f);
                    uint64_t sum = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            float w0, w1;
                            unpack_f2(add_f2(pack_f2(x[r][i][e], x[r][i][e + 1]), b2), w0, w1);
                            const uint64_t w2 = pack_f2(ex2(w0), ex2(w1));
                            sum = add_f2(sum, w2);
                            unpack_f2(add_f2(w2, one), w0, w1);      // the integer in the mantissa's low bits
                            w[e] = __float_as_uint(w0);
                            w[e + 1] = __float_as_uint(w1);
                        }
                        // digit k of tokens g, g + 8 of row 2 t, then of row 2 t + 1
                        const uint32_t p0 = __byte_perm(w[0], w[2], 0x5140), p1 = __byte_perm(w[1], w[3], 0x5140);
                        const uint32_t h0 = __byte_perm(w[0], w[2], 0x0062), h1 = __byte_perm(w[1], w[3], 0x0062);
                        pd[r][0][i] = __byte_perm(movm(__byte_perm(p0, p1, 0x5410)), 0, 0x3120);
                        pd[r][1][i] = __byte_perm(movm(__byte_perm(p0, p1, 0x7632)), 0, 0x3120);
                        pd[r][2][i] = __byte_perm(movm(__byte_perm(h0, h1, 0x5410)), 0, 0x3120);
                    }
                    float l[2];
                    unpack_f2(sum, l[0], l[1]);
#pragma unroll
                    for (int e = 0; e < 2; ++e)                      // tokens that are not seen take nothing from the page's scale (which may be NaN)
                        st.l[r][e] = st.l[r][e] * corr[r][e] + (l[e] == 0.f ? 0.f : l[e] * to[r][e] * iv);
                }
                if (__any_sync(~0u, moved)) {
#pragma unroll
                    for (int r = 0; r < RN; ++r)
#pragma unroll
                        for (int d = 0; d < D / 16; ++d)
#pragma unroll
                            for (int e = 0; e < 4; ++e) st.o[r][d][e] *= corr[r][e & 1];
                }
#pragma unroll
                for (int pn = 0; pn < kPanels; ++pn) {
                    const unsigned char* vp = wait(f0 + kPanels + pn) + g * kKvPage + 16 * t;
                    seen_words = 0;
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        const uint4 u = *reinterpret_cast<const uint4*>(vp + 16 * d * kKvPage);
                        const uint4 v = *reinterpret_cast<const uint4*>(vp + (16 * d + 8) * kKvPage);
                        const uint32_t a0[4] = {u.x, v.x, u.y, v.y}, a1[4] = {u.z, v.z, u.w, v.w};
                        seen_words |= u.w | v.w;
#pragma unroll
                        for (int r = 0; r < RN; ++r) {
                            int sum[3][4];
#pragma unroll
                            for (int j = 0; j < 3; ++j) {
                                mma_s8u8(sum[j], a0, pd[r][j][0], pd[r][j][1], sums0);
                                mma_s8u8(sum[j], a1, pd[r][j][2], pd[r][j][3], sum[j]);
                            }
                            float* o = st.o[r][4 * pn + d];
                            const uint64_t to2 = pack_f2(to[r][0], to[r][1]);
#pragma unroll
                            for (int e = 0; e < 4; e += 2)
                                unpack_f2(fma_f2(join_f2(sum[2] + e, sum[1] + e, sum[0] + e), to2, pack_f2(o[e], o[e + 1])), o[e], o[e + 1]);
                        }
                    }
                    arrived(seen_words);
                    fetch(f0 + kPanels + pn + depth);
                }
            }
        }
        // The incomplete last page, fp16: 16 tokens to a warp, staged with cp.async
        // in rows of 16-byte chunks c at c ^ (row % 8); tokens past the end are zero.
        if (tails) {
            constexpr int kCh = D / 8;                               // 16-byte chunks of a row
            const uint32_t kb = smem_u32(ring), vb = kb + 16 * D * 2;
            unsigned char* vp = ring + 16 * D * 2;
#pragma unroll
            for (int i = lane; i < 16 * kCh; i += 32) {
                const int r = i / kCh, c = i % kCh;
                const uint32_t n = warp * 16 + r < ntok ? 16u : 0u, to = (uint32_t)((r * kCh + (c ^ (r & 7))) * 16);
                const int64_t from = tail + (int64_t)(warp * 16 + r) * D + 8 * c;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(kb + to), "l"(a.c.k_tail + from), "r"(n) : "memory");
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(vb + to), "l"(a.c.v_tail + from), "r"(n) : "memory");
            }
            // Q as fp16 B fragments: panel p, step q: dimensions 64 p + 16 t + 4 q .. + 3 of query row 8 r + g
            uint32_t qf[RN][kPanels][4][2];
#pragma unroll
            for (int r = 0; r < RN; ++r) {
                const int row = row0 + 8 * r + g;
                const uint16_t* q = a.Q + (int64_t)(s.q0 + row / a.G) * a.ldQ + (int64_t)(h * a.G + row % a.G) * D + 16 * t;
#pragma unroll
                for (int p = 0; p < kPanels; ++p) {
                    const uint4 u = ldcg_128_if(q + 64 * p, row < rows), v = ldcg_128_if(q + 64 * p + 8, row < rows);
                    qf[r][p][0][0] = u.x;
                    qf[r][p][0][1] = u.y;
                    qf[r][p][1][0] = u.z;
                    qf[r][p][1][1] = u.w;
                    qf[r][p][2][0] = v.x;
                    qf[r][p][2][1] = v.y;
                    qf[r][p][3][0] = v.z;
                    qf[r][p][3][1] = v.w;
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
            float x[RN][4];
#pragma unroll
            for (int r = 0; r < RN; ++r) x[r][0] = x[r][1] = x[r][2] = x[r][3] = 0.f;
#pragma unroll
            for (int pn = 0; pn < kPanels; ++pn) {
                const int c0 = 8 * pn + 2 * t;                       // rows g and g + 8 (the same swizzle)
                const uint4 u0 = *reinterpret_cast<const uint4*>(ring + (g * kCh + (c0 ^ g)) * 16);
                const uint4 u1 = *reinterpret_cast<const uint4*>(ring + (g * kCh + ((c0 + 1) ^ g)) * 16);
                const uint4 v0 = *reinterpret_cast<const uint4*>(ring + ((g + 8) * kCh + (c0 ^ g)) * 16);
                const uint4 v1 = *reinterpret_cast<const uint4*>(ring + ((g + 8) * kCh + ((c0 + 1) ^ g)) * 16);
                const uint32_t af[4][4] = {{u0.x, v0.x, u0.y, v0.y}, {u0.z, v0.z, u0.w, v0.w}, {u1.x, v1.x, u1.y, v1.y}, {u1.z, v1.z, u1.w, v1.w}};
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int r = 0; r < RN; ++r) mma_16816(x[r], af[q], qf[r][pn][q]);
            }
            // A value that is not finite makes NaN of the rows that see its token and
            // must not reach the others (0 x inf): it is taken out of the product and
            // its token's scores become NaN instead.  The others' largest magnitude
            // gives the tokens the power of two that brings it to 64 .. 128, as codes
            // are, so that their weights share codes' range (2^-k plays s_V's part).  It is below 1 where the
            // largest passes 2^7: values 2^-21 of it and below then lose low bits.
            uint32_t poison = 0;
            __half2 am = __half2half2(__ushort_as_half(0));
            for (int i = lane; i < 16 * kCh; i += 32) {
                uint4* q = reinterpret_cast<uint4*>(vp + i * 16);
                uint32_t v[4] = {q->x, q->y, q->z, q->w};
                bool hit = false;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool l = (v[e] & 0x7c00u) == 0x7c00u, u = (v[e] & 0x7c000000u) == 0x7c000000u;
                    if (l) v[e] &= 0xffff0000u;
                    if (u) v[e] &= 0x0000ffffu;
                    hit |= l || u;
                    am = __hmax2(am, __habs2(u32_as_h2(v[e])));
                }
                if (hit) {
                    *q = make_uint4(v[0], v[1], v[2], v[3]);
                    poison |= 1u << (i / kCh);
                }
            }
            uint32_t ex = max(h2_as_u32(am) & 0x7c00u, (h2_as_u32(am) >> 16) & 0x7c00u) >> 10;   // biased by 15
            for (int o = 16; o > 0; o >>= 1) {
                poison |= __shfl_xor_sync(~0u, poison, o);
                ex = max(ex, __shfl_xor_sync(~0u, ex, o));
            }
            const int k2 = min(15, 21 - (int)ex);                    // -9 .. 15: 2^k2 is a normal fp16
            const __half2 up = __half2half2(__ushort_as_half((unsigned short)((k2 + 15) << 10)));
            __syncwarp();
            if (poison) {
#pragma unroll
                for (int r = 0; r < RN; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if ((poison >> (g + 8 * (e >> 1))) & 1) x[r][e] = __int_as_float(0x7fffffff);
            }
            int lim[RN][2];
#pragma unroll
            for (int r = 0; r < RN; ++r)
#pragma unroll
                for (int e = 0; e < 2; ++e) lim[r][e] = min(limit[r][e] - full * kKvPage, ntok - 1) - warp * 16;
            uint32_t pf[RN][2][2];
            softmax_tail<D, RN>(st, x, lim, a.scale_log2, (float)-k2, exp2f((float)k2), g, pf);
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
                // four 8 x 8 matrices: dimensions 16 d .. + 7 and + 8 .. + 15 of tokens 0 .. 7, then of tokens 8 .. 15
                const int r = (lane & 7) + (lane >> 4) * 8, c = 2 * d + ((lane >> 3) & 1);
                uint32_t v[4];
                ldsm4t(vb + (uint32_t)((r * kCh + (c ^ (r & 7))) * 16), v);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = h2_as_u32(__hmul2(u32_as_h2(v[e]), up));
#pragma unroll
                for (int q = 0; q < RN; ++q) {
                    mma_16816(st.o[q][d], v, pf[q][0]);
                    mma_16816(st.o[q][d], v, pf[q][1]);
                }
            }
        }
        if (tails) from = min(from, full * kKvPage + warp * 16);
        // ---- the warps' results: [warp][rows][D + 4] over the rings, m and l beside them ----
#pragma unroll
        for (int r = 0; r < RN; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (limit[r][e] >= from) st.m[r][e] = fmaxf(st.m[r][e], kLeastScore);
#pragma unroll
        for (int r = 0; r < RN; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                for (int o = 4; o < 32; o <<= 1) st.l[r][e] += __shfl_xor_sync(~0u, st.l[r][e], o);
        __syncthreads();
        float* all = reinterpret_cast<float*>(sm);
#pragma unroll
        for (int r = 0; r < RN; ++r) {
            float* so = all + (warp * kRows + 8 * r + 2 * t) * kPart + g;
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
                so[16 * d] = st.o[r][d][0];
                so[kPart + 16 * d] = st.o[r][d][1];
                so[16 * d + 8] = st.o[r][d][2];
                so[kPart + 16 * d + 8] = st.o[r][d][3];
            }
            if (g == 0) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    sml[(warp * kRows + 8 * r + 2 * t + e) * 2] = st.m[r][e];
                    sml[(warp * kRows + 8 * r + 2 * t + e) * 2 + 1] = st.l[r][e];
                }
            }
        }
        __syncthreads();
        const bool whole = pa == 0 && pe == w.pages;
        auto store = [&](int r, int c, float m, float l, const float4& o) {
            const int row = row0 + r;
            if (row >= rows) return;
            // a row that sees nothing is zero, one whose scores are all -inf NaN
            const float inv = l != 0.f ? 1.f / l : m == -INFINITY ? 0.f : __int_as_float(0x7fffffff);
            uint2 y;
            y.x = h2_as_u32(__floats2half2_rn(o.x * inv, o.y * inv));
            y.y = h2_as_u32(__floats2half2_rn(o.z * inv, o.w * inv));
            *reinterpret_cast<uint2*>(a.Y + (int64_t)(s.q0 + row / a.G) * a.ldY + (int64_t)(h * a.G + row % a.G) * D + 4 * c) = y;
        };
        // a part that starts its unit is its block's last, every other one its block's first
        float* part = a.partial + ((int64_t)blockIdx.x * 2 + (pa == 0)) * kRows * kPart;
#pragma unroll 1
        for (int i = tid; i < kRows * D / 4; i += kAttnThreads) {
            const int r = i / (D / 4), c = i % (D / 4);
            float m = -INFINITY, l = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kAttnWarps; ++k) m = fmaxf(m, sml[(k * kRows + r) * 2]);
            const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int k = 0; k < kAttnWarps; ++k) {
                const float f = ex2(sml[(k * kRows + r) * 2] - ref);
                const float4 v = *reinterpret_cast<const float4*>(all + (k * kRows + r) * kPart + 4 * c);
                l = fmaf(f, sml[(k * kRows + r) * 2 + 1], l);
                o = make_float4(fmaf(f, v.x, o.x), fmaf(f, v.y, o.y), fmaf(f, v.z, o.z), fmaf(f, v.w, o.w));
            }
            if (whole) {
                store(r, c, m, l, o);
            } else {
                __stcg(reinterpret_cast<float4*>(part + r * kPart + 4 * c), o);
                if (c == 0) __stcg(reinterpret_cast<float2*>(part + r * kPart + D), make_float2(m, l));
            }
        }
        if (!whole) {
            const long long u0 = lo - at + kAttnUnitCost;                // the unit's first page in the row of all
            const int first = (int)(u0 / per), parts = (int)((u0 + w.pages - 1) / per) - first + 1;
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                unsigned int prev;
                asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(prev) : "l"(a.tickets + first) : "memory");
                last_part = prev == (unsigned)(parts - 1);
                if (last_part) atomicExch(a.tickets + first, 0u);    // every part has counted: ready for the next call
            }
            __syncthreads();
            if (last_part) {
                __threadfence();
                auto of = [&](int k) { return a.partial + ((int64_t)(first + k) * 2 + (k == 0)) * kRows * kPart; };
                // every part's m, then its factor 2^(m - max), [part][row] over the rings; the rows' l
                for (int i = tid; i < parts * kRows; i += kAttnThreads) {
                    const float2 ml = __ldcg(reinterpret_cast<const float2*>(of(i / kRows) + (i % kRows) * kPart + D));
                    all[2 * i] = ml.x;
                    all[2 * i + 1] = ml.y;
                }
                __syncthreads();
                for (int r = warp; r < kRows; r += kAttnWarps) {
                    float m = -INFINITY, l = 0.f;
                    for (int k = lane; k < parts; k += 32) m = fmaxf(m, all[2 * (k * kRows + r)]);
                    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
                    const float ref = m == -INFINITY ? 0.f : m;
                    for (int k = lane; k < parts; k += 32) {
                        const float f = ex2(all[2 * (k * kRows + r)] - ref);
                        all[2 * (k * kRows + r)] = f;
                        l = fmaf(f, all[2 * (k * kRows + r) + 1], l);
                    }
                    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
                    if (lane == 0) {
                        sml[2 * r] = m;
                        sml[2 * r + 1] = l;
                    }
                }
                __syncthreads();
                // a warp adds every fourth part, eight rows at a time, two parts' loads in flight; then the warps' sums
                constexpr int kLoads = D / 16;                       // 16-byte words of a lane: 8 rows of D / 4 words in 32 lanes
                float* sums = all + 2 * (kAttnParts + 2) * kRows;    // [warp][rows][D], behind the factors
#pragma unroll 1
                for (int r0 = 0; r0 < kRows; r0 += 8) {
                    float4 o[kLoads];
#pragma unroll
                    for (int i = 0; i < kLoads; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
                    for (int k = warp; k < parts; k += 2 * kAttnWarps) {
                        uint4 v[2][kLoads];
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int i = 0; i < kLoads; ++i) {
                                const int word = lane + 32 * i, kk = k + u * kAttnWarps;
                                v[u][i] = ldcg_128_if(of(kk) + (r0 + word / (D / 4)) * kPart + word % (D / 4) * 4, kk < parts);
                            }
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int i = 0; i < kLoads; ++i) {
                                const int kk = min(k + u * kAttnWarps, parts - 1);
                                const float f = all[2 * (kk * kRows + r0 + (lane + 32 * i) / (D / 4))];
                                o[i] = make_float4(fmaf(f, __uint_as_float(v[u][i].x), o[i].x), fmaf(f, __uint_as_float(v[u][i].y), o[i].y),
                                                   fmaf(f, __uint_as_float(v[u][i].z), o[i].z), fmaf(f, __uint_as_float(v[u][i].w), o[i].w));
                            }
                    }
#pragma unroll
                    for (int i = 0; i < kLoads; ++i)
                        reinterpret_cast<float4*>(sums)[(warp * kRows + r0) * (D / 4) + lane + 32 * i] = o[i];
                }
                __syncthreads();
                for (int i = tid; i < kRows * D / 4; i += kAttnThreads) {
                    float4 o = reinterpret_cast<const float4*>(sums)[i];
#pragma unroll
                    for (int k = 1; k < kAttnWarps; ++k) {
                        const float4 v = reinterpret_cast<const float4*>(sums)[k * kRows * (D / 4) + i];
                        o = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
                    }
                    store(i / (D / 4), i % (D / 4), sml[i / (D / 4) * 2], sml[i / (D / 4) * 2 + 1], o);
                }
            }
        }
        lo += take;
        off += take;
        if (lo < hi) {                                               // the rings are filled again by bulk copies
            fence_proxy_async_all();
            __syncthreads();
        }
    }
}

static int attn_rows(int64_t rows) { return rows <= 8 ? 8 : 16; }
static size_t attn_smem(int rows) { return (size_t)kAttnWarps * 16384 + kAttnWarps * rows * 2 * sizeof(float); }

KvAttnPlan plan_kv_attention(const KvBatchView& b, int G, int kv_heads, int head_dim, int num_sms) {
    KvAttnPlan p = {};
    const int64_t rows = (int64_t)b.max_new * G, heads = (int64_t)b.n_seq * kv_heads, P = b.max_pages;
    // Here 16 rows and a page take 3.6 ns of the whole GPU, beside 30 us for the
    // start and the joins; attention_tc.cu takes 256 rows to a block, whatever rows
    // stay empty, and expects its own time.  8 kv heads and 32768 tokens: 64 rows of
    // one sequence 84 us here, 126 there, 128 rows 139 and 109; of eight sequences 918
    // and 396; after 2048 tokens 107 and 45.  Below 64 rows this kernel is faster but
    // for a few us.
    const KvTcShares tc = kv_tc_shares(b, G, kv_heads, num_sms);
    p.S = tc.S;
    p.tc = rows >= 64 && tc.us <= 0.0036 * heads * ((rows + 15) / 16) * P + 30.;
    p.rows = attn_rows(rows);
    // the blocks that are resident, or as many as there can be shares
    const int64_t units = (int64_t)b.n_seq * kv_heads * ((rows + p.rows - 1) / p.rows);
    const int64_t want = (units * ((b.max_pages > 0 ? b.max_pages : 1) + kAttnUnitCost) + kAttnLeastShare - 1) / kAttnLeastShare;
    p.sms = num_sms;
    p.blocks = num_sms * (p.rows == 8 ? 3 : 2);
    if (p.blocks > want) p.blocks = (int)want;
    p.partial_bytes = p.tc ? kv_tc_partial_bytes(b, G, kv_heads, p.S, head_dim) : (size_t)p.blocks * 2 * p.rows * (head_dim + 4) * sizeof(float);
    return p;
}

template <int D, int RN>
static cudaError_t launch_attn(const KvAttnArgs& a, int blocks, cudaStream_t st) {
    const void* f = (const void*)kv_attention_kernel<D, RN>;
    static SmemLimit limit;
    cudaError_t e = limit.raise(f, (int)attn_smem(8 * RN));
    if (e != cudaSuccess) return e;
    void* args[] = {(void*)&a};
    return launch_pdl(f, (unsigned)blocks, kAttnThreads, attn_smem(8 * RN), st, args);
}

cudaError_t launch_kv_attention(const KvCacheView& c, const KvBatchView& b, const uint16_t* Q, int64_t ldQ, int q_heads,
                                float scale, uint16_t* Y, int64_t ldY, unsigned int* tickets, float* partial,
                                const KvAttnPlan& p, cudaStream_t st) {
    if (p.tc) return launch_kv_attention_tc(c, b, Q, ldQ, q_heads, scale, Y, ldY, tickets, partial, p.S, st);
    KvAttnArgs a = {c, b, Q, Y, ldQ, ldY, scale * 1.44269504088896340736f, q_heads / c.kv_heads, p.sms, partial, tickets,
                    device_status_ptr()};
    if (c.head_dim == 64) return p.rows == 8 ? launch_attn<64, 1>(a, p.blocks, st) : launch_attn<64, 2>(a, p.blocks, st);
    return p.rows == 8 ? launch_attn<128, 1>(a, p.blocks, st) : launch_attn<128, 2>(a, p.blocks, st);
}

}  // namespace glowq
