// kvcache.cu -- the paged 8-bit key/value cache: append with the position
// rotation applied on the way, and reading back what is stored.
//
// A page holds 64 consecutive tokens of a sequence.  A complete page is stored
// in 8-bit integers with one scale per kv head for its keys and one for its
// values; the tokens of a sequence's incomplete last page are kept in fp16 in
// the sequence's tail until the page completes.  So each code is rounded once,
// with the scale of the whole page, and what the cache holds depends on the
// tokens alone, not on how they were cut into appends.
#include "common.cuh"
#include "internal.cuh"
#include "kvcache.cuh"
#include "quant8.cuh"

namespace glowq {

constexpr int kAppendThreads = 256;

struct KvAppendArgs {
    KvCacheView c;
    KvBatchView b;
    const uint16_t *Q, *K, *V;
    uint16_t* Q_out;
    const float* rope;       // [rope_len][D]: cosines of the D/2 pairs, then sines; nullptr: no rotation
    int64_t ldQ, ldK, ldV, ldQo;
    int G;                   // query heads per kv head (0: no queries)
    int rope_len;
    int npg;                 // pages that max_new tokens may touch
    unsigned int* status;
};

// Elements [8 i, 8 i + 8) and the same behind the middle of a head's row.
struct HalfRow {
    uint4 lo, hi;
};
__device__ __forceinline__ HalfRow load_row_if(const uint16_t* p, int i, int half, bool there) {
    return {ldcg_128_if(p + 8 * i, there), ldcg_128_if(p + half + 8 * i, there)};
}
__device__ __forceinline__ void store_row(uint16_t* p, int i, int half, const HalfRow& v) {
    *reinterpret_cast<uint4*>(p + 8 * i) = v.lo;
    *reinterpret_cast<uint4*>(p + half + 8 * i) = v.hi;
}
// Cosines and sines of the eight pairs (8 i + e, D/2 + 8 i + e) at one position.
struct Turn {
    float4 c[2], s[2];
};
__device__ __forceinline__ Turn load_turn(const float* cs, int i, int half) {
    const float4 *c = reinterpret_cast<const float4*>(cs + 8 * i), *s = reinterpret_cast<const float4*>(cs + half + 8 * i);
    return {{__ldg(c), __ldg(c + 1)}, {__ldg(s), __ldg(s + 1)}};
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t n) {   // n 16 or 0: then zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Pairs (x_i, x_{i + D/2}) turned by the position's angle: two fp32 products and
// one sum each, unfused, rounded to fp16 once.
__device__ __forceinline__ void rotate(HalfRow& v, const Turn& t) {
    const uint32_t a[4] = {v.lo.x, v.lo.y, v.lo.z, v.lo.w}, b[4] = {v.hi.x, v.hi.y, v.hi.z, v.hi.w};
    const float c[8] = {t.c[0].x, t.c[0].y, t.c[0].z, t.c[0].w, t.c[1].x, t.c[1].y, t.c[1].z, t.c[1].w};
    const float s[8] = {t.s[0].x, t.s[0].y, t.s[0].z, t.s[0].w, t.s[1].x, t.s[1].y, t.s[1].z, t.s[1].w};
    uint32_t x[4], y[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float2 f = __half22float2(u32_as_h2(a[q])), h = __half22float2(u32_as_h2(b[q]));
        x[q] = h2_as_u32(__floats2half2_rn(__fsub_rn(__fmul_rn(f.x, c[2 * q]), __fmul_rn(h.x, s[2 * q])),
                                           __fsub_rn(__fmul_rn(f.y, c[2 * q + 1]), __fmul_rn(h.y, s[2 * q + 1]))));
        y[q] = h2_as_u32(__floats2half2_rn(__fadd_rn(__fmul_rn(h.x, c[2 * q]), __fmul_rn(f.x, s[2 * q])),
                                           __fadd_rn(__fmul_rn(h.y, c[2 * q + 1]), __fmul_rn(f.y, s[2 * q + 1]))));
    }
    v = {make_uint4(x[0], x[1], x[2], x[3]), make_uint4(y[0], y[1], y[2], y[3])};
}
// A page's value codes on their way through shared memory: [D][64 tokens] in
// words of four tokens, word w of row d at w ^ (d / 8 % 16) (eight dimensions
// and a few tokens are moved at a time: no more than two lanes meet in a bank).
template <int D>
struct CodeTile {
    uint32_t w[D][kKvPage / 4];
    __device__ __forceinline__ uint32_t& at(int d, int i) { return w[d][i ^ ((d >> 3) & 15)]; }
    // the 16 tokens from 16 c of row d
    __device__ __forceinline__ uint4 chunk(int d, int c) {
        const int f = (d >> 3) & 15;
        uint4 v = *reinterpret_cast<const uint4*>(&w[d][4 * (c ^ (f >> 2))]);
        if (f & 1) v = make_uint4(v.y, v.x, v.w, v.z);
        if (f & 2) v = make_uint4(v.z, v.w, v.x, v.y);
        return v;
    }
    __device__ __forceinline__ void set_chunk(int d, int c, uint4 v) {
        const int f = (d >> 3) & 15;
        if (f & 1) v = make_uint4(v.y, v.x, v.w, v.z);
        if (f & 2) v = make_uint4(v.z, v.w, v.x, v.y);
        *reinterpret_cast<uint4*>(&w[d][4 * (c ^ (f >> 2))]) = v;
    }
};
// 4 x 4 bytes: byte j of r[i] and byte i of r[j] change places.
__device__ __forceinline__ void transpose4(uint32_t (&r)[4]) {
    const uint32_t a = __byte_perm(r[0], r[1], 0x5140), b = __byte_perm(r[2], r[3], 0x5140);
    const uint32_t c = __byte_perm(r[0], r[1], 0x7362), d = __byte_perm(r[2], r[3], 0x7362);
    r[0] = __byte_perm(a, b, 0x5410);
    r[1] = __byte_perm(a, b, 0x7632);
    r[2] = __byte_perm(c, d, 0x5410);
    r[3] = __byte_perm(c, d, 0x7632);
}
// The same across four lanes S apart, each with one row: lane t gets byte t of all four.
template <int S>
__device__ __forceinline__ uint32_t transpose4_lanes(uint32_t w, int t) {
    const uint32_t a = __shfl_xor_sync(~0u, w, S);
    w = __byte_perm(w, a, t & 1 ? 0x3715 : 0x6240);      // bytes (t & 1) and (t & 1) + 2 of both lanes, the even lane's first
    const uint32_t b = __shfl_xor_sync(~0u, w, 2 * S);
    return __byte_perm(w, b, t & 2 ? 0x3276 : 0x5410);
}

// One block: one page that the step touches, of one sequence and kv head (and
// the query heads that share it).  The block of the first touched page also
// takes the last one when that stays incomplete: it reads the old tail for the
// first and writes the new tail for the last, in this order.
// The rows of a page wait in shared memory, each thread's own, so that all of a
// block's loads are in flight and registers leave room for three blocks an SM
// (held in registers: two; six prompts of 40 heads took 63 us instead of 58); blocks of one page's heads
// are neighbours, whose rows are neighbours in memory; a key and its queries
// share their angles.  168 MB (4096 tokens of 32 heads of 128) in 45 us, 56 % of
// the copy bandwidth: what is left is latency, the chain from the sequence's
// numbers to its rows and to the codes (issue slots 55 %, DRAM 37 % busy).
template <int D>
__global__ void __launch_bounds__(kAppendThreads, 3) kv_append_kernel(const __grid_constant__ KvAppendArgs a) {
    constexpr int kHalf = D / 2, kItems = D / 16;        // items of 8 + 8 elements per row
    constexpr int kPer = kKvPage * kItems / kAppendThreads;
    extern __shared__ __align__(16) uint4 stage[];
    __shared__ float red[2][kAppendThreads / 32];
    __shared__ __align__(16) CodeTile<D> vt;
    pdl_wait();
    pdl_launch_dependents();
    const int h = blockIdx.x % a.c.kv_heads, bj = blockIdx.x / a.c.kv_heads, j = bj % a.npg, b = bj / a.npg;
    const KvSeq s = kv_sequence(a.b, b);
    if (s.nq == 0 && s.ok) return;
    const bool bad = !s.ok || s.start < 0 || s.slot < 0 || s.slot >= a.c.slots || s.len > (int64_t)a.b.max_pages * kKvPage ||
                     (a.rope && s.len > a.rope_len);
    if (bad) {
        if (threadIdx.x == 0) record_status(a.status, GLOWQ_ERR_INDEX);
        return;
    }
    const int p0 = s.start / kKvPage, p1 = (s.len - 1) / kKvPage;
    const bool open = s.len % kKvPage != 0;              // the last page stays incomplete
    if (p0 + j > p1 || (j > 0 && p0 + j == p1 && open)) return;
    const int64_t tail = ((int64_t)s.slot * a.c.kv_heads + h) * kKvPage * D;
    const int tid = threadIdx.x, i = tid % kItems;

    for (int p = p0 + j;; p = p1) {
        if ((p + 1) * (int64_t)kKvPage > s.len) {        // stays incomplete: K, V and queries of its new tokens
            const int t0 = max(s.start, p * kKvPage), n = (s.len - t0) * kItems;
            int lw = 3;                                  // threads over (token, item): 2^lw; the others take other heads
            while (lw < 8 && (1 << lw) < n) ++lw;
            for (int it = tid & ((1 << lw) - 1); it < n; it += 1 << lw) {
                const int pos = t0 + it / kItems;
                const int64_t row = s.q0 + (pos - s.start), to = tail + (int64_t)(pos % kKvPage) * D;
                auto source = [&](int g) {               // heads of the group: queries, K, V
                    return g < a.G   ? a.Q + row * a.ldQ + (int64_t)(h * a.G + g) * D
                           : g == a.G ? a.K + row * a.ldK + (int64_t)h * D
                                      : a.V + row * a.ldV + (int64_t)h * D;
                };
                const int step = kAppendThreads >> lw;
                int g = tid >> lw;
                HalfRow next = load_row_if(source(g), i, kHalf, g < a.G + 2);
                Turn turn;
                if (a.rope) turn = load_turn(a.rope + (int64_t)pos * D, i, kHalf);
                for (; g < a.G + 2; g += step) {
                    HalfRow v = next;
                    next = load_row_if(source(g + step), i, kHalf, g + step < a.G + 2);
                    if (a.rope && g <= a.G) rotate(v, turn);
                    store_row(g < a.G   ? a.Q_out + row * a.ldQo + (int64_t)(h * a.G + g) * D
                              : g == a.G ? a.c.k_tail + to
                                         : a.c.v_tail + to,
                              i, kHalf, v);
                }
            }
        } else {
            // a thread's own rows wait in shared memory: [K, V, query][q][half][thread]
            auto slot = [&](int what, int q) { return &stage[((what * kPer + q) * 2) * kAppendThreads + tid]; };
            auto fetch = [&](int what, int q, const uint16_t* src, bool there) {
                const uint32_t dst = smem_u32(slot(what, q)), n = there ? 16u : 0u;
                cp_async16(dst, src + 8 * i, n);
                cp_async16(dst + kAppendThreads * 16, src + kHalf + 8 * i, n);
            };
            auto get = [&](int what, int q) { return HalfRow{slot(what, q)[0], slot(what, q)[kAppendThreads]}; };
            const int page = ldcg_s32(a.b.table + (int64_t)b * a.b.max_pages + p);
#pragma unroll
            for (int q = 0; q < kPer; ++q) {
                const int tok = (tid + q * kAppendThreads) / kItems, pos = p * kKvPage + tok;
                const int64_t row = s.q0 + (pos - s.start), from = tail + (int64_t)tok * D;
                const bool old = pos < s.start;
                fetch(0, q, old ? a.c.k_tail + from : a.K + row * a.ldK + (int64_t)h * D, true);
                fetch(1, q, old ? a.c.v_tail + from : a.V + row * a.ldV + (int64_t)h * D, true);
                if (a.G > 0) fetch(2, q, a.Q + row * a.ldQ + (int64_t)h * a.G * D, !old);
            }
            __half2 kam = __half2half2(__ushort_as_half(0)), vam = kam;
            for (int q = 0; q < kPer; ++q) {
                const int pos = p * kKvPage + (tid + q * kAppendThreads) / kItems;
                const bool old = pos < s.start;
                const int64_t row = s.q0 + (pos - s.start);
                Turn turn;
                if (a.rope) turn = load_turn(a.rope + (int64_t)pos * D, i, kHalf);
                cp_async_wait_all();
                HalfRow x = get(0, q);
                if (a.rope && !old) {
                    rotate(x, turn);
                    slot(0, q)[0] = x.lo;
                    slot(0, q)[kAppendThreads] = x.hi;
                }
                amax8(x.lo, kam);
                amax8(x.hi, kam);
                x = get(1, q);
                amax8(x.lo, vam);
                amax8(x.hi, vam);
                if (old) continue;
                for (int g = 0; g < a.G; ++g) {
                    const int64_t at = (int64_t)(h * a.G + g) * D;
                    cp_async_wait_all();
                    x = get(2, q);
                    if (g + 1 < a.G) fetch(2, q, a.Q + row * a.ldQ + at + D, true);
                    if (a.rope) rotate(x, turn);
                    store_row(a.Q_out + row * a.ldQo + at, i, kHalf, x);
                }
            }
            for (int o = 16; o > 0; o >>= 1) {
                kam = __hmax2_nan(kam, __shfl_xor_sync(~0u, kam, o));
                vam = __hmax2_nan(vam, __shfl_xor_sync(~0u, vam, o));
            }
            if ((tid & 31) == 0) {
                red[0][tid >> 5] = amax_float(kam);
                red[1][tid >> 5] = amax_float(vam);
            }
            __syncthreads();
            float ka = 0.f, va = 0.f;
            bool kf = true, vf = true;
#pragma unroll
            for (int w = 0; w < kAppendThreads / 32; ++w) {
                ka = fmaxf(ka, red[0][w]);
                va = fmaxf(va, red[1][w]);
                kf &= red[0][w] <= 65504.f;
                vf &= red[1][w] <= 65504.f;
            }
            // 2^-24 is fp16's smallest value: the scale of an all-zero page, below every other
            const float nan = __int_as_float(0x7fffffff);
            const float ks = kf ? __fdiv_rn(fmaxf(ka, 5.9604644775390625e-8f), 127.f) : nan;
            const float vs = vf ? __fdiv_rn(fmaxf(va, 5.9604644775390625e-8f), 127.f) : nan;
            const float kinv = __fdiv_rn(1.f, ks), vinv = __fdiv_rn(1.f, vs);
            if (page < 0 || page >= a.c.pages) {
                if (tid == 0) record_status(a.status, GLOWQ_ERR_INDEX);
            } else {
                const int64_t ph = (int64_t)page * a.c.kv_heads + h;
                int8_t* kc = a.c.k_codes + ph * kKvPage * D;
                uint4* vc = reinterpret_cast<uint4*>(a.c.v_codes + ph * kKvPage * D);
                if (tid == 0) {
                    a.c.k_scales[ph] = ks;
                    a.c.v_scales[ph] = vs;
                }
                for (int q = 0; q < kPer; ++q) {
                    const int tok = (tid + q * kAppendThreads) / kItems;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {        // dimensions 8 i .. + 7 and the same behind the middle
                        const int dim = e * kHalf + 8 * i;
                        *reinterpret_cast<uint2*>(kc + ((dim >> 6) * kKvPage + tok) * 64 + (dim & 63)) =
                            kf ? codes8(slot(0, q)[e * kAppendThreads], ks, kinv) : make_uint2(0u, 0u);
                        const uint2 c = vf ? codes8(slot(1, q)[e * kAppendThreads], vs, vinv) : make_uint2(0u, 0u);
                        // four tokens' lanes trade bytes: a word of four tokens of one dimension each
                        vt.at(dim + (tok & 3), tok >> 2) = transpose4_lanes<kItems>(c.x, tok & 3);
                        vt.at(dim + 4 + (tok & 3), tok >> 2) = transpose4_lanes<kItems>(c.y, tok & 3);
                    }
                }
                __syncthreads();
                for (int it = tid; it < D * 4; it += kAppendThreads) vc[it] = vt.chunk(it >> 2, it & 3);
            }
        }
        if (j > 0 || p == p1 || !open) return;
        __syncthreads();                                 // the old tail is read before the new one is written
    }
}

// ---------------------------------------------------------------------------
// Values at positions [first, first + count) of every sequence, fp16:
// fp16_RN(code * scale) of complete pages, the tail's values, zero at and
// behind the sequence's end.
// ---------------------------------------------------------------------------
struct KvReadArgs {
    KvCacheView c;
    KvBatchView b;
    const int* first;        // nullptr: 0
    int count, npg;
    uint16_t *K, *V;         // [n_seq][count][kv_heads][D]
    unsigned int* status;
};

// fp16_RN(code * s) of a word's four codes: a byte with its sign bit turned is
// 128 + q, placed in 2^23's mantissa.
__device__ __forceinline__ uint2 values4(uint32_t w, float s) {
    const uint32_t u = w ^ 0x80808080u;
    auto f = [&](uint32_t sel) { return __fmul_rn(__uint_as_float(__byte_perm(u, 0x4b000000u, sel)) - 8388736.f, s); };
    return make_uint2(h2_as_u32(__floats2half2_rn(f(0x7540), f(0x7541))), h2_as_u32(__floats2half2_rn(f(0x7542), f(0x7543))));
}
// One block: one page's part of a sequence and kv head.  A thread takes eight
// dimensions of four tokens: codes of V are by dimension, and change places in
// its registers.
template <int D>
__global__ void __launch_bounds__(2 * D) kv_read_kernel(const __grid_constant__ KvReadArgs a) {
    constexpr int kChunks = D / 8;
    __shared__ __align__(16) CodeTile<D> vt;
    pdl_wait();
    pdl_launch_dependents();
    const int h = blockIdx.x % a.c.kv_heads, bj = blockIdx.x / a.c.kv_heads, j = bj % a.npg, b = bj / a.npg, tid = threadIdx.x;
    const int len = ldcg_s32(a.b.kv_len + b), slot = ldcg_s32(a.b.slot + b), asked = a.first ? ldcg_s32(a.first + b) : 0;
    bool ok = asked >= 0 && asked <= kKvReadMax && len >= 0 && len <= (int64_t)a.b.max_pages * kKvPage;
    const int first = ok ? asked : 0;                    // (count <= kKvReadMax: no position passes 2^31)
    const int p = first / kKvPage + j;
    const int t0 = max(first, p * kKvPage), t1 = min(first + a.count, (p + 1) * kKvPage);
    if (t0 >= t1) return;
    const bool complete = (p + 1) * kKvPage <= len;
    int page = 0;
    if (ok && p * kKvPage < len) {
        if (complete) {
            page = ldcg_s32(a.b.table + (int64_t)b * a.b.max_pages + p);
            ok = page >= 0 && page < a.c.pages;
        } else {
            ok = slot >= 0 && slot < a.c.slots;
        }
    }
    if (!ok && tid == 0) record_status(a.status, GLOWQ_ERR_INDEX);
    const int64_t ph = (int64_t)page * a.c.kv_heads + h, tail = ((int64_t)slot * a.c.kv_heads + h) * kKvPage * D;
    const int c = tid % kChunks, dim = 8 * c;
    auto put = [&](int pos, const uint4& k, const uint4& v) {
        const int64_t to = (((int64_t)b * a.count + (pos - first)) * a.c.kv_heads + h) * D + dim;
        *reinterpret_cast<uint4*>(a.K + to) = k;
        *reinterpret_cast<uint4*>(a.V + to) = v;
    };
    if (ok && complete) {
        const int t4 = tid / kChunks;                    // tokens 4 t4 .. + 3 (2 D threads: all 64)
        const uint4* vc = reinterpret_cast<const uint4*>(a.c.v_codes + ph * kKvPage * D);
        const int8_t* kc = a.c.k_codes + ph * kKvPage * D + ((dim >> 6) * kKvPage + 4 * t4) * 64 + (dim & 63);
        const uint4 v0 = ldcg_128(vc + tid), v1 = ldcg_128(vc + tid + 2 * D);
        uint2 k[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) k[e] = ldcg_64(kc + e * 64);
        const float ks = ldcg_f32(a.c.k_scales + ph), vs = ldcg_f32(a.c.v_scales + ph);
        vt.set_chunk(tid >> 2, tid & 3, v0);
        vt.set_chunk((tid + 2 * D) >> 2, tid & 3, v1);
        __syncthreads();
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            lo[e] = vt.at(dim + e, t4);
            hi[e] = vt.at(dim + 4 + e, t4);
        }
        transpose4(lo);
        transpose4(hi);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int pos = p * kKvPage + 4 * t4 + e;
            const uint2 ka = values4(k[e].x, ks), kb = values4(k[e].y, ks), va = values4(lo[e], vs), vb = values4(hi[e], vs);
            if (pos >= t0 && pos < t1) put(pos, make_uint4(ka.x, ka.y, kb.x, kb.y), make_uint4(va.x, va.y, vb.x, vb.y));
        }
        return;
    }
    for (int pos = t0 + tid / kChunks; pos < t1; pos += 2 * D / kChunks) {
        const int64_t at = tail + (int64_t)(pos - p * kKvPage) * D + dim;
        const bool there = ok && pos < len;
        const uint4 k = ldcg_128_if(a.c.k_tail + at, there), v = ldcg_128_if(a.c.v_tail + at, there);
        put(pos, k, v);
    }
}

cudaError_t launch_kv_append(const KvCacheView& c, const KvBatchView& b, const uint16_t* Q, int64_t ldQ, int q_heads,
                             const uint16_t* K, int64_t ldK, const uint16_t* V, int64_t ldV, const float* rope,
                             int rope_len, uint16_t* Q_out, int64_t ldQo, cudaStream_t st) {
    KvAppendArgs a = {c, b, Q, K, V, Q_out, rope, ldQ, ldK, ldV, ldQo, Q ? q_heads / c.kv_heads : 0, rope_len, 0,
                      device_status_ptr()};
    a.npg = kv_touched_pages(b.max_new);
    const unsigned grid = (unsigned)((int64_t)a.npg * c.kv_heads * b.n_seq);
    void* args[] = {(void*)&a};
    const void* f = c.head_dim == 64 ? (const void*)kv_append_kernel<64> : (const void*)kv_append_kernel<128>;
    const int smem = 3 * kKvPage * c.head_dim * 2;       // keys, values and one query head of a page
    static SmemLimit limits[2];
    cudaError_t e = limits[c.head_dim == 128].raise(f, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(f, grid, kAppendThreads, smem, st, args);
}

cudaError_t launch_kv_read(const KvCacheView& c, const KvBatchView& b, const int* first, int count, uint16_t* K,
                           uint16_t* V, cudaStream_t st) {
    KvReadArgs a = {c, b, first, count, kv_touched_pages(count), K, V, device_status_ptr()};
    const unsigned grid = (unsigned)((int64_t)a.npg * c.kv_heads * b.n_seq);
    void* args[] = {(void*)&a};
    return launch_pdl(c.head_dim == 64 ? (const void*)kv_read_kernel<64> : (const void*)kv_read_kernel<128>, grid,
                      2 * c.head_dim, 0, st, args);
}

}  // namespace glowq
