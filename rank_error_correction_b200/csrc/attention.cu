// attention.cu -- causal attention of a step's queries over the paged 8-bit
// key/value cache.
//
//   o_i = sum_j softmax_j(scale q_i . k_j) v_j,   j <= len - n + i  (n new rows)
//
// Codes enter the products as the exact integers they are; the page's scales
// meet them in fp32: s_K on the scores, and s_V inside the exponent, as
//   w_ij = 2^(x_ij + log2 s_V - m_i),  x_ij = scale log2(e) s_K q_i . k_j
// with m_i the running maximum of x + log2 s_V.  The numerator is then
// sum_j w_ij v_j with integer v, and the denominator sum_pages (sum_j w_ij) / s_V,
// so that weights stay in fp16's range however the pages' scales differ.
// Weights are scaled by 2^8 (the factor cancels): fp16's smallest normal is
// then 2^-22 of the largest weight.  One rounding of w to fp16 (2^-11), sums,
// maxima and outputs in fp32.
#include "common.cuh"
#include "internal.cuh"
#include "kvcache.cuh"

namespace glowq {

constexpr int kAttnWarps = 4;
constexpr int kAttnRing = 3;             // half-pages (K or V of one page) in flight per warp
constexpr float kWeightExp = 8.f;

struct KvAttnArgs {
    KvCacheView c;
    KvBatchView b;
    const uint16_t* Q;
    uint16_t* Y;
    int64_t ldQ, ldY;
    float scale_log2;        // scale log2(e)
    int G, rt, S;
    float* partial;          // [((b Hkv + h) rt + tile) S + s][16][D + 2]
    unsigned int* tickets;   // [(b Hkv + h) rt + tile], zero between calls
    unsigned int* status;
};

__device__ __forceinline__ void attn_bulk(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    mbar_arrive_expect_tx(bar, bytes);
    bulk_g2s(dst, src, bytes, bar);
}
// Four int8 codes as fp16 pairs, exactly: bytes with the sign bit turned are 128 + q, placed in 1024's mantissa.
__device__ __forceinline__ void cvt_codes(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = w ^ 0x80808080u;
    const __half2 bias = u32_as_h2(0x64806480u);         // 1152
    lo = h2_as_u32(__hsub2(u32_as_h2(__byte_perm(u, 0x64646464u, 0x4140)), bias));
    hi = h2_as_u32(__hsub2(u32_as_h2(__byte_perm(u, 0x64646464u, 0x4342)), bias));
}
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

// Running softmax of a warp's 16 rows: this lane's rows g and g + 8.
template <int D>
struct AttnState {
    float m[2], l[2], o[D / 8][4];
};

// One tile of 64 columns.  x: scores in the C-fragment layout of eight 16 x 8
// tiles; col(j, e): the token (within the page) of column 2 t + e of tile j;
// lim: last visible token of each row relative to the page; lv = log2 s_V.
// Returns the weights as A fragments.
template <int D, class Col>
__device__ __forceinline__ void softmax_tile(AttnState<D>& st, float (&x)[8][4], const int (&lim)[2], float xs, float lv,
                                             float inv_sv, bool masked, Col col, uint32_t (&pf)[8][2]) {
    float mx[2] = {st.m[0], st.m[1]};
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float v = fmaf(x[j][e], xs, lv);
            if (masked && col(j, e & 1) > lim[e >> 1]) v = -INFINITY;
            x[j][e] = v;
            mx[e >> 1] = fmaxf(mx[e >> 1], v);
        }
    float base[2], corr[2], sum[2] = {0.f, 0.f};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(~0u, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(~0u, mx[r], 2));
        const float ref = mx[r] == -INFINITY ? 0.f : mx[r];   // nothing visible yet: weights 2^-inf = 0
        corr[r] = ex2(st.m[r] - ref);
        st.m[r] = mx[r];
        base[r] = ref - kWeightExp;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w[e] = ex2(x[j][e] - base[e >> 1]);
            sum[e >> 1] += w[e];
        }
        pf[j][0] = h2_as_u32(__floats2half2_rn(w[0], w[1]));
        pf[j][1] = h2_as_u32(__floats2half2_rn(w[2], w[3]));
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        sum[r] += __shfl_xor_sync(~0u, sum[r], 1);
        sum[r] += __shfl_xor_sync(~0u, sum[r], 2);
        // rows that see nothing of the page take nothing from its scale (which may be NaN)
        st.l[r] = st.l[r] * corr[r] + (sum[r] == 0.f ? 0.f : sum[r] * inv_sv);
    }
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) st.o[n][e] *= corr[e >> 1];
}

// One block: 16 rows (row = new token i and query head gq of the kv head's
// group, i G + gq) of one sequence and kv head, over share s of the pages.
// Its warps take the pages in turn, each with a ring of K and V halves filled
// by bulk copies; lane (g, t) feeds the MMA 16 consecutive bytes of a row at a
// time (k in the order 16 t + 4 step, the same in both operands).  The warps'
// results meet in shared memory, the shares' in the workspace: the share that
// counts last adds them in share order.
template <int D>
__global__ void __launch_bounds__(kAttnWarps * 32) kv_attention_kernel(const __grid_constant__ KvAttnArgs a) {
    constexpr int kHalfPage = kKvPage * D;               // bytes of a page's K (or V) of one head
    constexpr int kPanels = D / 64;
    extern __shared__ __align__(128) unsigned char sm[];
    // [4 warps][ring of 3 half-pages] (later the warps' outputs), [16][D] queries, m / l, barriers
    uint16_t* sq = reinterpret_cast<uint16_t*>(sm + kAttnWarps * kAttnRing * kHalfPage);
    float* sml = reinterpret_cast<float*>(sq + 16 * D);  // [warps][16][2]
    uint64_t* bars = reinterpret_cast<uint64_t*>(sml + kAttnWarps * 32);
    __shared__ int last_share;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int share = blockIdx.x % a.S, tile = (blockIdx.x / a.S) % a.rt;
    const int bh = blockIdx.x / a.S / a.rt, h = bh % a.c.kv_heads, b = bh / a.c.kv_heads;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kAttnWarps * kAttnRing; ++i) mbar_init(bars + i, 1);
        fence_mbar_init();
    }
    pdl_wait();
    pdl_launch_dependents();
    const KvSeq s = kv_sequence(a.b, b);
    const int rows = s.nq * a.G, row0 = tile * 16;
    if (!s.ok && threadIdx.x == 0) record_status(a.status, GLOWQ_ERR_INDEX);
    if (row0 >= rows) return;
    // a length that the table or the tails cannot hold: nothing is visible, and the rows are zero
    const bool tailed = s.len % kKvPage != 0;
    const bool bad = s.len > (int64_t)a.b.max_pages * kKvPage || (tailed && (s.slot < 0 || s.slot >= a.c.slots));
    if (bad && threadIdx.x == 0) record_status(a.status, GLOWQ_ERR_INDEX);
    const int last_tok = (min(row0 + 15, rows - 1)) / a.G;           // the tile's last new token
    const int seen = bad ? 0 : max(0, s.start + last_tok + 1);       // tokens that the tile sees
    const int npages = (seen + kKvPage - 1) / kKvPage;
    const int per = (npages + a.S - 1) / a.S;
    const int pa = min(npages, share * per), pb = min(npages, pa + per);
    const int full = s.len / kKvPage;                                // pages held in codes
    const int pc = min(pb, full);                                    // ... of this share: [pa, pc); a tail page may follow

    for (int i = threadIdx.x; i < 16 * D / 8; i += kAttnWarps * 32) {
        const int r = i / (D / 8), row = row0 + r;
        reinterpret_cast<uint4*>(sq)[i] =
            ldcg_128_if(a.Q + (int64_t)(s.q0 + row / a.G) * a.ldQ + (int64_t)(h * a.G + row % a.G) * D + (i % (D / 8)) * 8, row < rows);
    }
    __syncthreads();
    // Q as A fragments: panel p, step q: dimensions 64 p + 16 t + 4 q .. + 3 of rows g and g + 8
    uint32_t qf[kPanels][4][4];
#pragma unroll
    for (int p = 0; p < kPanels; ++p)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint2 u = *reinterpret_cast<const uint2*>(sq + g * D + 64 * p + 16 * t + 4 * q);
            const uint2 v = *reinterpret_cast<const uint2*>(sq + (g + 8) * D + 64 * p + 16 * t + 4 * q);
            qf[p][q][0] = u.x;
            qf[p][q][1] = v.x;
            qf[p][q][2] = u.y;
            qf[p][q][3] = v.y;
        }
    int limit[2];                                                    // last visible position of rows g, g + 8
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = row0 + g + 8 * r;
        limit[r] = row < rows ? s.start + row / a.G : -1;
    }
    const int least = s.start + row0 / a.G;                          // smallest limit of the tile's rows
    const bool short_tile = row0 + 16 > rows;

    AttnState<D> st;
    st.m[0] = st.m[1] = -INFINITY;
    st.l[0] = st.l[1] = 0.f;
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) st.o[n][e] = 0.f;

    unsigned char* ring = sm + warp * kAttnRing * kHalfPage;
    uint64_t* wbar = bars + warp * kAttnRing;
    const int* table = a.b.table + (int64_t)b * a.b.max_pages;
    // half-pages in the order K, V of this warp's pages; the next one to fetch
    int fp = pa + warp, fh = 0, fs = 0;
    auto fetch = [&]() {
        if (fp < pc) {
            const int page = ldcg_s32(table + fp);
            if (lane == 0 && page >= 0 && page < a.c.pages) {
                const int64_t at = ((int64_t)page * a.c.kv_heads + h) * kHalfPage;
                attn_bulk(smem_u32(ring + fs * kHalfPage), (fh ? a.c.v_codes : a.c.k_codes) + at, kHalfPage, wbar + fs);
            }
            if (fh) fp += kAttnWarps;
            fh ^= 1;
        }
        if (++fs == kAttnRing) fs = 0;
    };
#pragma unroll
    for (int i = 0; i < kAttnRing; ++i) fetch();
    int cs = 0;
    uint32_t phases = 0;                                             // bit i: parity of ring entry i
    bool ok = true;
    for (int p = pa + warp; p < pc; p += kAttnWarps) {
        const int page = ldcg_s32(table + p);
        const bool there = page >= 0 && page < a.c.pages;            // (else nothing was fetched: the page is skipped)
        if (!there) {
            if (lane == 0) record_status(a.status, GLOWQ_ERR_INDEX);
            for (int i = 0; i < 2; ++i) {
                if (++cs == kAttnRing) cs = 0;
                fetch();
            }
            continue;
        }
        const int64_t ph = (int64_t)page * a.c.kv_heads + h;
        const float ks = ldcg_f32(a.c.k_scales + ph), vs = ldcg_f32(a.c.v_scales + ph);
        float x[8][4];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j][0] = x[j][1] = x[j][2] = x[j][3] = 0.f;
        if (ok) ok = mbar_wait(wbar + cs, (phases >> cs) & 1, a.status);
        phases ^= 1u << cs;
        const unsigned char* kp = ring + cs * kHalfPage;
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int pn = 0; pn < kPanels; ++pn) {
                const uint4 w = *reinterpret_cast<const uint4*>(kp + (pn * kKvPage + 16 * (g >> 1) + 2 * j + (g & 1)) * 64 + 16 * t);
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t bf[2];
                    cvt_codes(ww[q], bf[0], bf[1]);
                    mma_16816(x[j], qf[pn][q], bf);
                }
            }
        __syncwarp();
        if (++cs == kAttnRing) cs = 0;
        fetch();
        const int lim[2] = {limit[0] - p * kKvPage, limit[1] - p * kKvPage};
        uint32_t pf[8][2];
        softmax_tile<D>(st, x, lim, ks * a.scale_log2, log2f(vs), 1.f / vs, short_tile || least < p * kKvPage + kKvPage - 1,
                        [&](int j, int e) { return 16 * t + 2 * j + e; }, pf);
        if (ok) ok = mbar_wait(wbar + cs, (phases >> cs) & 1, a.status);
        phases ^= 1u << cs;
        const unsigned char* vp = ring + cs * kHalfPage;
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
            const uint4 w = *reinterpret_cast<const uint4*>(vp + (8 * n + g) * kKvPage + 16 * t);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t bf[2];
                cvt_codes(ww[q], bf[0], bf[1]);
                const uint32_t af[4] = {pf[2 * q][0], pf[2 * q][1], pf[2 * q + 1][0], pf[2 * q + 1][1]};
                mma_16816(st.o[n], af, bf);
            }
        }
        __syncwarp();
        if (++cs == kAttnRing) cs = 0;
        fetch();
    }
    // The incomplete last page, fp16, by the warp whose turn it is: keys and then
    // values staged with cp.async in rows of 16-byte chunks c at c ^ (row % 8);
    // tokens past the end are zero.
    if (pc < pb && (pc - pa) % kAttnWarps == warp) {
        const int ntok = s.len - full * kKvPage;
        const int64_t tail = ((int64_t)s.slot * a.c.kv_heads + h) * kHalfPage;
        constexpr int kCh = D / 8;                                   // 16-byte chunks of a row
        const uint32_t rb = smem_u32(ring);
        auto stage = [&](const uint16_t* src) {
            for (int i = lane; i < kKvPage * kCh; i += 32) {
                const int r = i / kCh, c = i % kCh;
                const uint32_t n = r < ntok ? 16u : 0u;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(rb + (uint32_t)((r * kCh + (c ^ (r & 7))) * 16)),
                             "l"(src + tail + (int64_t)r * D + 8 * c), "r"(n)
                             : "memory");
            }
            asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
            __syncwarp();
        };
        stage(a.c.k_tail);
        float x[8][4];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j][0] = x[j][1] = x[j][2] = x[j][3] = 0.f;
            const int r = 8 * j + g;
#pragma unroll
            for (int pn = 0; pn < kPanels; ++pn) {
                const int c0 = 8 * pn + 2 * t;
                const uint4 u = *reinterpret_cast<const uint4*>(ring + (r * kCh + (c0 ^ (r & 7))) * 16);
                const uint4 v = *reinterpret_cast<const uint4*>(ring + (r * kCh + ((c0 + 1) ^ (r & 7))) * 16);
                const uint32_t b0[2] = {u.x, u.y}, b1[2] = {u.z, u.w}, b2[2] = {v.x, v.y}, b3[2] = {v.z, v.w};
                mma_16816(x[j], qf[pn][0], b0);
                mma_16816(x[j], qf[pn][1], b1);
                mma_16816(x[j], qf[pn][2], b2);
                mma_16816(x[j], qf[pn][3], b3);
            }
        }
        __syncwarp();
        stage(a.c.v_tail);
        // A value that is not finite makes NaN of the rows that see its token and
        // must not reach the others (0 x inf): it is taken out of the product and
        // its token's scores become NaN instead.  The others' largest magnitude
        // gives the tail the power of two that brings it to 64 .. 128, as codes
        // are, so that its weights share their range (2^-k plays s_V's part).
        uint64_t poison = 0;
        __half2 am = __half2half2(__ushort_as_half(0));
        for (int i = lane; i < kKvPage * kCh; i += 32) {
            const int r = i / kCh;
            uint4* q = reinterpret_cast<uint4*>(ring + i * 16);
            uint32_t w[4] = {q->x, q->y, q->z, q->w};
            bool hit = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool l = (w[e] & 0x7c00u) == 0x7c00u, u = (w[e] & 0x7c000000u) == 0x7c000000u;
                if (l) w[e] &= 0xffff0000u;
                if (u) w[e] &= 0x0000ffffu;
                hit |= l || u;
                am = __hmax2(am, __habs2(u32_as_h2(w[e])));
            }
            if (hit) {
                *q = make_uint4(w[0], w[1], w[2], w[3]);
                poison |= 1ull << r;
            }
        }
        uint32_t ex = max(h2_as_u32(am) & 0x7c00u, (h2_as_u32(am) >> 16) & 0x7c00u) >> 10;   // biased by 15
        for (int o = 16; o > 0; o >>= 1) {
            poison |= __shfl_xor_sync(~0u, poison, o);
            ex = max(ex, __shfl_xor_sync(~0u, ex, o));
        }
        const int k2 = min(15, 21 - (int)ex);                        // -9 .. 15: 2^k2 is a normal fp16
        const __half2 up = __half2half2(__ushort_as_half((unsigned short)((k2 + 15) << 10)));
        __syncwarp();
        if (poison) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if ((poison >> (8 * j + 2 * t + (e & 1))) & 1) x[j][e] = __int_as_float(0x7fffffff);
        }
        const int lim[2] = {min(limit[0] - full * kKvPage, ntok - 1), min(limit[1] - full * kKvPage, ntok - 1)};
        uint32_t pf[8][2];
        softmax_tile<D>(st, x, lim, a.scale_log2, (float)-k2, exp2f((float)k2), true, [&](int j, int e) { return 8 * j + 2 * t + e; }, pf);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t af[4] = {pf[2 * q][0], pf[2 * q][1], pf[2 * q + 1][0], pf[2 * q + 1][1]};
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
                // four 8 x 8 matrices: tokens 16 q .. + 7 and + 8 .. + 15 of dimensions 16 n .. + 7, then of + 8 .. + 15
                const int r = 16 * q + (lane & 15), c = 2 * n + (lane >> 4);
                uint32_t v[4];
                ldsm4t(rb + (uint32_t)((r * kCh + (c ^ (r & 7))) * 16), v);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = h2_as_u32(__hmul2(u32_as_h2(v[e]), up));
                const uint32_t b0[2] = {v[0], v[1]}, b1[2] = {v[2], v[3]};
                mma_16816(st.o[2 * n], af, b0);
                mma_16816(st.o[2 * n + 1], af, b1);
            }
        }
    }
    // ---- the warps' results: [warp][16][D] over the rings, m and l beside them ----
    __syncthreads();
    float* so = reinterpret_cast<float*>(sm) + warp * 16 * D;
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
        *reinterpret_cast<float2*>(so + g * D + 8 * n + 2 * t) = make_float2(st.o[n][0], st.o[n][1]);
        *reinterpret_cast<float2*>(so + (g + 8) * D + 8 * n + 2 * t) = make_float2(st.o[n][2], st.o[n][3]);
    }
    if (t == 0) {
        sml[(warp * 16 + g) * 2] = st.m[0];
        sml[(warp * 16 + g) * 2 + 1] = st.l[0];
        sml[(warp * 16 + g + 8) * 2] = st.m[1];
        sml[(warp * 16 + g + 8) * 2 + 1] = st.l[1];
    }
    __syncthreads();
    const int64_t unit = (int64_t)bh * a.rt + tile;
    float* part = a.partial + unit * a.S * 16 * (D + 2);
    // parts of one row, in order: each with its own m, l and outputs
    auto merge = [&](int n, auto m_of, auto l_of, auto o_of, float& m, float& l, float4& o) {
        m = -INFINITY;
        l = 0.f;
        o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < n; ++w) m = fmaxf(m, m_of(w));
        const float ref = m == -INFINITY ? 0.f : m;
        for (int w = 0; w < n; ++w) {
            const float lw = l_of(w), f = ex2(m_of(w) - ref);
            if (lw == 0.f) continue;                                 // saw nothing (a NaN part stays: f NaN is NaN, 0 NaN too)
            const float4 p = o_of(w);
            l = fmaf(f, lw, l);
            o.x = fmaf(f, p.x, o.x);
            o.y = fmaf(f, p.y, o.y);
            o.z = fmaf(f, p.z, o.z);
            o.w = fmaf(f, p.w, o.w);
        }
    };
    auto store = [&](int r, int c, float l, const float4& o) {
        const int row = row0 + r;
        if (row >= rows) return;
        const float inv = l == 0.f ? 0.f : 1.f / l;                  // a row that sees nothing is zero
        uint2 y;
        y.x = h2_as_u32(__floats2half2_rn(o.x * inv, o.y * inv));
        y.y = h2_as_u32(__floats2half2_rn(o.z * inv, o.w * inv));
        *reinterpret_cast<uint2*>(a.Y + (int64_t)(s.q0 + row / a.G) * a.ldY + (int64_t)(h * a.G + row % a.G) * D + 4 * c) = y;
    };
    for (int i = threadIdx.x; i < 16 * D / 4; i += kAttnWarps * 32) {
        const int r = i / (D / 4), c = i % (D / 4);
        float m, l;
        float4 o;
        merge(kAttnWarps, [&](int w) { return sml[(w * 16 + r) * 2]; }, [&](int w) { return sml[(w * 16 + r) * 2 + 1]; },
              [&](int w) { return *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(sm) + (w * 16 + r) * D + 4 * c); },
              m, l, o);
        if (a.S == 1) {
            store(r, c, l, o);
        } else {
            float* q = part + (share * 16 + r) * (D + 2);
            __stcg(reinterpret_cast<float2*>(q + 4 * c), make_float2(o.x, o.y));
            __stcg(reinterpret_cast<float2*>(q + 4 * c + 2), make_float2(o.z, o.w));
            if (c == 0) __stcg(reinterpret_cast<float2*>(q + D), make_float2(m, l));
        }
    }
    if (a.S == 1) return;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        unsigned int prev;
        asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(prev) : "l"(a.tickets + unit) : "memory");
        last_share = prev == (unsigned)(a.S - 1);
        if (last_share) atomicExch(a.tickets + unit, 0u);            // every share has counted: ready for the next call
    }
    __syncthreads();
    if (!last_share) return;
    __threadfence();
    for (int i = threadIdx.x; i < 16 * D / 4; i += kAttnWarps * 32) {
        const int r = i / (D / 4), c = i % (D / 4);
        float m, l;
        float4 o;
        const float* q = part + r * (D + 2);
        const int step = 16 * (D + 2);
        merge(a.S, [&](int w) { return __ldcg(q + w * step + D); }, [&](int w) { return __ldcg(q + w * step + D + 1); },
              [&](int w) {
                  const float2 u = __ldcg(reinterpret_cast<const float2*>(q + w * step + 4 * c));
                  const float2 v = __ldcg(reinterpret_cast<const float2*>(q + w * step + 4 * c + 2));
                  return make_float4(u.x, u.y, v.x, v.y);
              },
              m, l, o);
        store(r, c, l, o);
    }
}

static size_t attn_smem(int D) {
    return (size_t)kAttnWarps * kAttnRing * kKvPage * D + 16 * D * 2 + kAttnWarps * 32 * 4 + kAttnWarps * kAttnRing * 8;
}

KvAttnPlan plan_kv_attention(const KvBatchView& b, int G, int kv_heads, int head_dim, int num_sms) {
    KvAttnPlan p;
    p.tc = (int64_t)b.max_new * G >= 64;
    p.rt = (int)(((int64_t)b.max_new * G + 15) / 16);
    const int64_t units = (int64_t)b.n_seq * kv_heads * p.rt;
    p.S = 1;
    if (units > 0 && units < 2 * num_sms) {
        int64_t S = 2 * num_sms / units;
        const int64_t most = b.max_pages / kAttnWarps;               // a page for each warp, at least
        if (S > most) S = most;
        if (S > 64) S = 64;
        if (S > 1) p.S = (int)S;
    }
    if (p.tc) p.S = 1;
    p.partial_bytes = p.S > 1 ? (size_t)units * p.S * 16 * (head_dim + 2) * sizeof(float) : 0;
    return p;
}

template <int D>
static cudaError_t launch_attn(const KvAttnArgs& a, unsigned grid, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute((const void*)kv_attention_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)attn_smem(D));
    if (e != cudaSuccess) return e;
    void* args[] = {(void*)&a};
    return launch_pdl((const void*)kv_attention_kernel<D>, grid, kAttnWarps * 32, attn_smem(D), st, args);
}

cudaError_t launch_kv_attention(const KvCacheView& c, const KvBatchView& b, const uint16_t* Q, int64_t ldQ, int q_heads,
                                float scale, uint16_t* Y, int64_t ldY, unsigned int* tickets, float* partial,
                                const KvAttnPlan& p, cudaStream_t st) {
    if (p.tc) return launch_kv_attention_tc(c, b, Q, ldQ, q_heads, scale, Y, ldY, st);
    KvAttnArgs a = {c, b, Q, Y, ldQ, ldY, scale * 1.44269504088896340736f, q_heads / c.kv_heads, p.rt, p.S, partial, tickets,
                    device_status_ptr()};
    const unsigned grid = (unsigned)((int64_t)b.n_seq * c.kv_heads * p.rt * p.S);
    return c.head_dim == 64 ? launch_attn<64>(a, grid, st) : launch_attn<128>(a, grid, st);
}

}  // namespace glowq
