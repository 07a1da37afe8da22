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
__device__ __forceinline__ HalfRow load_row(const uint16_t* p, int i, int half) {
    return {ldcg_128(p + 8 * i), ldcg_128(p + half + 8 * i)};
}
__device__ __forceinline__ void store_row(uint16_t* p, int i, int half, const HalfRow& v) {
    *reinterpret_cast<uint4*>(p + 8 * i) = v.lo;
    *reinterpret_cast<uint4*>(p + half + 8 * i) = v.hi;
}
// Pairs (x_i, x_{i + D/2}) turned by the position's angle: two fp32 products and
// one sum each, unfused, rounded to fp16 once.
__device__ __forceinline__ HalfRow rotate(const HalfRow& v, const float* cs, int i, int half) {
    const uint32_t a[4] = {v.lo.x, v.lo.y, v.lo.z, v.lo.w}, b[4] = {v.hi.x, v.hi.y, v.hi.z, v.hi.w};
    uint32_t x[4], y[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float2 c = __ldg(reinterpret_cast<const float2*>(cs + 8 * i) + q);
        const float2 s = __ldg(reinterpret_cast<const float2*>(cs + half + 8 * i) + q);
        const float2 f = __half22float2(u32_as_h2(a[q])), h = __half22float2(u32_as_h2(b[q]));
        x[q] = h2_as_u32(__floats2half2_rn(__fsub_rn(__fmul_rn(f.x, c.x), __fmul_rn(h.x, s.x)),
                                           __fsub_rn(__fmul_rn(f.y, c.y), __fmul_rn(h.y, s.y))));
        y[q] = h2_as_u32(__floats2half2_rn(__fadd_rn(__fmul_rn(h.x, c.x), __fmul_rn(f.x, s.x)),
                                           __fadd_rn(__fmul_rn(h.y, c.y), __fmul_rn(f.y, s.y))));
    }
    return {make_uint4(x[0], x[1], x[2], x[3]), make_uint4(y[0], y[1], y[2], y[3])};
}
// One block: one page that the step touches, of one sequence and kv head (and
// the query heads that share it).  The block of the first touched page also
// takes the last one when that stays incomplete: it reads the old tail for the
// first and writes the new tail for the last, in this order.
template <int D>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const __grid_constant__ KvAppendArgs a) {
    constexpr int kHalf = D / 2, kItems = D / 16;        // items of 8 + 8 elements per row
    constexpr int kPer = kKvPage * kItems / kAppendThreads;
    __shared__ float red[2][kAppendThreads / 32];
    __shared__ __align__(16) unsigned char vt[D][kKvPage + 16];   // codes of V by dimension
    pdl_wait();
    pdl_launch_dependents();
    const int j = blockIdx.x % a.npg, bh = blockIdx.x / a.npg;
    const int h = bh % a.c.kv_heads, b = bh / a.c.kv_heads;
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
    const int tid = threadIdx.x;

    for (int p = p0 + j;; p = p1) {
        const int t0 = max(s.start, p * kKvPage), t1 = min(s.len, (p + 1) * kKvPage);   // new tokens of the page
        // queries
        if (a.G > 0) {
            const int n = (t1 - t0) * a.G * kItems;
            for (int it = tid; it < n; it += kAppendThreads) {
                const int i = it % kItems, rg = it / kItems, gq = rg % a.G, pos = t0 + rg / a.G;
                const int64_t row = s.q0 + (pos - s.start);
                HalfRow v = load_row(a.Q + row * a.ldQ + (int64_t)(h * a.G + gq) * D, i, kHalf);
                if (a.rope) v = rotate(v, a.rope + (int64_t)pos * D, i, kHalf);
                store_row(a.Q_out + row * a.ldQo + (int64_t)(h * a.G + gq) * D, i, kHalf, v);
            }
        }
        const bool complete = (p + 1) * kKvPage <= s.len;
        if (!complete) {
            const int n = (t1 - t0) * kItems;
            for (int it = tid; it < n; it += kAppendThreads) {
                const int i = it % kItems, pos = t0 + it / kItems;
                const int64_t row = s.q0 + (pos - s.start), to = tail + (int64_t)(pos % kKvPage) * D;
                HalfRow k = load_row(a.K + row * a.ldK + (int64_t)h * D, i, kHalf);
                if (a.rope) k = rotate(k, a.rope + (int64_t)pos * D, i, kHalf);
                store_row(a.c.k_tail + to, i, kHalf, k);
                store_row(a.c.v_tail + to, i, kHalf, load_row(a.V + row * a.ldV + (int64_t)h * D, i, kHalf));
            }
        } else {
            HalfRow k[kPer], v[kPer];
            __half2 kam = __half2half2(__ushort_as_half(0)), vam = kam;
#pragma unroll
            for (int q = 0; q < kPer; ++q) {
                const int it = tid + q * kAppendThreads, i = it % kItems, pos = p * kKvPage + it / kItems;
                if (pos < s.start) {
                    const int64_t from = tail + (int64_t)(pos % kKvPage) * D;
                    k[q] = load_row(a.c.k_tail + from, i, kHalf);
                    v[q] = load_row(a.c.v_tail + from, i, kHalf);
                } else {
                    const int64_t row = s.q0 + (pos - s.start);
                    k[q] = load_row(a.K + row * a.ldK + (int64_t)h * D, i, kHalf);
                    v[q] = load_row(a.V + row * a.ldV + (int64_t)h * D, i, kHalf);
                    if (a.rope) k[q] = rotate(k[q], a.rope + (int64_t)pos * D, i, kHalf);
                }
                amax8(k[q].lo, kam);
                amax8(k[q].hi, kam);
                amax8(v[q].lo, vam);
                amax8(v[q].hi, vam);
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
            const int page = ldcg_s32(a.b.table + (int64_t)b * a.b.max_pages + p);
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
#pragma unroll
                for (int q = 0; q < kPer; ++q) {
                    const int it = tid + q * kAppendThreads, i = it % kItems, tok = it / kItems;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {        // dimensions 8 i .. + 7 and the same behind the middle
                        const int dim = e * kHalf + 8 * i;
                        *reinterpret_cast<uint2*>(kc + ((dim >> 6) * kKvPage + tok) * 64 + (dim & 63)) =
                            kf ? codes8(e ? k[q].hi : k[q].lo, ks, kinv) : make_uint2(0u, 0u);
                        const uint2 c = vf ? codes8(e ? v[q].hi : v[q].lo, vs, vinv) : make_uint2(0u, 0u);
#pragma unroll
                        for (int r = 0; r < 8; ++r)
                            vt[dim + r][tok] = (unsigned char)((r < 4 ? c.x >> (8 * r) : c.y >> (8 * (r - 4))) & 255u);
                    }
                }
                __syncthreads();
                for (int it = tid; it < D * 4; it += kAppendThreads)
                    vc[it] = *reinterpret_cast<const uint4*>(&vt[it >> 2][(it & 3) * 16]);
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

template <int D>
__global__ void __launch_bounds__(256) kv_read_kernel(const __grid_constant__ KvReadArgs a) {
    constexpr int kChunks = D / 8;
    __shared__ __align__(16) unsigned char vt[D][kKvPage + 16];
    pdl_wait();
    pdl_launch_dependents();
    const int j = blockIdx.x % a.npg, bh = blockIdx.x / a.npg;
    const int h = bh % a.c.kv_heads, b = bh / a.c.kv_heads, tid = threadIdx.x;
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
    const bool codes = ok && complete;
    float ks = 0.f, vs = 0.f;
    if (codes) {
        ks = ldcg_f32(a.c.k_scales + ph);
        vs = ldcg_f32(a.c.v_scales + ph);
        const uint4* vc = reinterpret_cast<const uint4*>(a.c.v_codes + ph * kKvPage * D);
        for (int it = tid; it < D * 4; it += 256) *reinterpret_cast<uint4*>(&vt[it >> 2][(it & 3) * 16]) = ldcg_128(vc + it);
        __syncthreads();
    }
    for (int it = tid; it < (t1 - t0) * kChunks; it += 256) {
        const int c = it % kChunks, pos = t0 + it / kChunks, tok = pos - p * kKvPage, dim = 8 * c;
        uint4 k = make_uint4(0, 0, 0, 0), v = k;
        if (codes) {
            const uint2 q = ldcg_64(a.c.k_codes + ph * kKvPage * D + ((dim >> 6) * kKvPage + tok) * 64 + (dim & 63));
            uint32_t ko[4], vo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t w = e < 2 ? q.x >> (16 * e) : q.y >> (16 * (e - 2));
                ko[e] = h2_as_u32(__floats2half2_rn((float)(int8_t)(w & 255) * ks, (float)(int8_t)((w >> 8) & 255) * ks));
                vo[e] = h2_as_u32(__floats2half2_rn((float)(int8_t)vt[dim + 2 * e][tok] * vs,
                                                    (float)(int8_t)vt[dim + 2 * e + 1][tok] * vs));
            }
            k = make_uint4(ko[0], ko[1], ko[2], ko[3]);
            v = make_uint4(vo[0], vo[1], vo[2], vo[3]);
        } else if (ok && pos < len) {
            k = ldcg_128(a.c.k_tail + tail + (int64_t)tok * D + dim);
            v = ldcg_128(a.c.v_tail + tail + (int64_t)tok * D + dim);
        }
        const int64_t to = (((int64_t)b * a.count + (pos - first)) * a.c.kv_heads + h) * D + dim;
        *reinterpret_cast<uint4*>(a.K + to) = k;
        *reinterpret_cast<uint4*>(a.V + to) = v;
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
    return launch_pdl(c.head_dim == 64 ? (const void*)kv_append_kernel<64> : (const void*)kv_append_kernel<128>, grid,
                      kAppendThreads, 0, st, args);
}

cudaError_t launch_kv_read(const KvCacheView& c, const KvBatchView& b, const int* first, int count, uint16_t* K,
                           uint16_t* V, cudaStream_t st) {
    KvReadArgs a = {c, b, first, count, kv_touched_pages(count), K, V, device_status_ptr()};
    const unsigned grid = (unsigned)((int64_t)a.npg * c.kv_heads * b.n_seq);
    void* args[] = {(void*)&a};
    return launch_pdl(c.head_dim == 64 ? (const void*)kv_read_kernel<64> : (const void*)kv_read_kernel<128>, grid, 256,
                      0, st, args);
}

}  // namespace glowq
