// int8.cu -- 8-bit integer weights and activations (W8A8): quantisers, and the
// corrected product for small T on warp-level integer MMAs.
//
//   s_t = max_k |x[t][k]| / 127,  c[t][k] = rint(x[t][k] / s_t)      per token
//   s_o = max_k |w[o][k]| / 127,  q[o][k] = rint(w[o][k] / s_o)      per output channel
//   y[t][o] = s_t s_o sum_k c[t][k] q[o][k] + sum_j R[t][j] A[o][j],  R = X B^T
//
// The integer sum is exact (d <= 131072 keeps it below 2^31), so no order of
// summation changes y; the scales and the correction meet it in fp32 and y is
// rounded to fp16 once.
#include <cfloat>

#include "common.cuh"
#include "internal.cuh"
#include "quant8.cuh"

namespace glowq {

// ---------------------------------------------------------------------------
// Quantisers.  All decisions in IEEE fp32 (division, rint to even).  A row
// that holds an infinity or a NaN gets the scale NaN and codes 0, so that
// everything computed from it is NaN, as the unquantised product would be.
// ---------------------------------------------------------------------------
constexpr int kQuantThreads = 256;

__device__ __forceinline__ float int8_row_scale(float amax, bool finite) {
    if (!finite) return __int_as_float(0x7fffffff);
    return amax > 0.f ? __fdiv_rn(amax, 127.f) : 1.f;
}
__device__ __forceinline__ int int8_code(float x, float s) {
    const float q = rintf(__fdiv_rn(x, s));
    return (int)fminf(fmaxf(q, -127.f), 127.f);   // NaN (scale NaN) -> -127, replaced by the caller
}
__device__ __forceinline__ uint32_t int8_pack4(float a, float b, float c, float d, float s) {
    return (uint32_t)(int8_code(a, s) & 255) | ((uint32_t)(int8_code(b, s) & 255) << 8) |
           ((uint32_t)(int8_code(c, s) & 255) << 16) | ((uint32_t)(int8_code(d, s) & 255) << 24);
}
// Maximum of |x| and whether every x is finite, over the block; the result in every thread.
__device__ __forceinline__ void block_amax(float& amax, bool& finite) {
    __shared__ float red[kQuantThreads / 32];
    __shared__ int bad[kQuantThreads / 32];
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
    const int b = __any_sync(~0u, !finite);
    if ((threadIdx.x & 31) == 0) {
        red[threadIdx.x >> 5] = amax;
        bad[threadIdx.x >> 5] = b;
    }
    __syncthreads();
    int anyb = 0;
    for (int i = 0; i < kQuantThreads / 32; ++i) {
        amax = fmaxf(amax, red[i]);
        anyb |= bad[i];
    }
    finite = !anyb;
}

// One weight row per block, read twice (the second time from L2).
__global__ void __launch_bounds__(kQuantThreads) pack_int8_kernel(const float* __restrict__ W, int64_t d,
                                                                  int8_t* __restrict__ codes,
                                                                  float* __restrict__ scales) {
    const int64_t o = blockIdx.x;
    const float4* w = reinterpret_cast<const float4*>(W + o * d);
    const int n4 = (int)(d / 4);
    float amax = 0.f;
    bool finite = true;
    for (int i = threadIdx.x; i < n4; i += kQuantThreads) {
        const float4 v = w[i];
        amax = fmaxf(fmaxf(fmaxf(amax, fabsf(v.x)), fmaxf(fabsf(v.y), fabsf(v.z))), fabsf(v.w));
        finite &= fabsf(v.x) <= FLT_MAX && fabsf(v.y) <= FLT_MAX && fabsf(v.z) <= FLT_MAX && fabsf(v.w) <= FLT_MAX;
    }
    block_amax(amax, finite);
    const float s = int8_row_scale(amax, finite);
    if (threadIdx.x == 0) scales[o] = s;
    uint32_t* out = reinterpret_cast<uint32_t*>(codes + o * d);
    for (int i = threadIdx.x; i < n4; i += kQuantThreads) {
        const float4 v = w[i];
        out[i] = finite ? int8_pack4(v.x, v.y, v.z, v.w, s) : 0u;
    }
}

__global__ void __launch_bounds__(256) dequant_int8_kernel(const int8_t* __restrict__ codes,
                                                           const float* __restrict__ scales, int64_t d,
                                                           __half* __restrict__ out) {
    const int64_t o = blockIdx.x;
    const float s = scales[o];
    for (int64_t k = threadIdx.x; k < d; k += 256) out[o * d + k] = __float2half_rn((float)codes[o * d + k] * s);
}

// Quantises token `t` of X by the whole block; store(i, v) receives the codes
// of elements 8 i .. 8 i + 7.  d % 8 == 0, rows 16-byte aligned.
template <class Store>
__device__ __forceinline__ void quantize_token(const uint16_t* __restrict__ X, int64_t t, int64_t d,
                                               float* __restrict__ scales, Store store) {
    const uint4* x = reinterpret_cast<const uint4*>(X + t * d);
    const int n8 = (int)(d / 8);
    constexpr int kKeep = 8;                 // the first 8 kKeep 256 elements of a row stay in registers
    uint4 keep[kKeep];
    __half2 am = __half2half2(__ushort_as_half(0));
#pragma unroll
    for (int j = 0; j < kKeep; ++j) {
        const int i = threadIdx.x + j * kQuantThreads;
        keep[j] = ldcg_128_if(x + i, i < n8);
    }
#pragma unroll
    for (int j = 0; j < kKeep; ++j) amax8(keep[j], am);
#pragma unroll 4
    for (int i = threadIdx.x + kKeep * kQuantThreads; i < n8; i += kQuantThreads) amax8(ldcg_128(x + i), am);
    float amax = amax_float(am);
    bool finite = amax <= 65504.f;
    block_amax(amax, finite);
    const float s = int8_row_scale(amax, finite);
    if (threadIdx.x == 0) scales[t] = s;
    const float inv = __fdiv_rn(1.f, s);
    auto code = [&](int i, const uint4& u) { store(i, finite ? codes8(u, s, inv) : make_uint2(0u, 0u)); };
#pragma unroll
    for (int j = 0; j < kKeep; ++j) {
        const int i = threadIdx.x + j * kQuantThreads;
        if (i < n8) code(i, keep[j]);
    }
#pragma unroll 4
    for (int i = threadIdx.x + kKeep * kQuantThreads; i < n8; i += kQuantThreads) code(i, ldcg_128(x + i));
}

// One token per block, codes row-major [T][d].
__global__ void __launch_bounds__(kQuantThreads) quantize_act_int8_kernel(const uint16_t* __restrict__ X, int64_t d,
                                                                          int8_t* __restrict__ codes,
                                                                          float* __restrict__ scales) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t t = blockIdx.x;
    uint2* out = reinterpret_cast<uint2*>(codes + t * d);
    quantize_token(X, t, d, scales, [&](int i, uint2 q) { out[i] = q; });
}
// This block's codes and scale are complete: count it, for a product that does
// not wait for the whole grid (a grid's end takes 1.5 us to reach the next).
__device__ __forceinline__ void count_ready(unsigned int* ready) {
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        flag_release_add(ready, 1u);
    }
}
// The same inside a forward call, counting the tokens done.  Behind the
// projection (!first), which has waited for X, it runs beside it; one block
// waits for its end, so that this grid's end implies both.
__global__ void __launch_bounds__(kQuantThreads) int8_quantize_kernel(const uint16_t* __restrict__ X, int64_t d,
                                                                      int8_t* __restrict__ codes,
                                                                      float* __restrict__ scales, unsigned int* ready,
                                                                      bool first) {
    if (first) pdl_wait();
    pdl_launch_dependents();
    const int64_t t = blockIdx.x;
    uint2* out = reinterpret_cast<uint2*>(codes + t * d);
    quantize_token(X, t, d, scales, [&](int i, uint2 q) { out[i] = q; });
    count_ready(ready);
    if (!first && t == 0) pdl_wait();
}

// ---------------------------------------------------------------------------
// Small T (<= 16), first launch.  The first blocks compute R = X B^T, two rows
// of B for all tokens per block, fp32 sums in a fixed order, rounded to fp16
// (splitting d over blocks as well costs more in joining the parts than it
// saves: 8.0 us against 4.9 at T = 1, d = 4096).  The others quantise a token
// each into the layout that the product stages with one bulk copy,
// [d/64][TOK][64] (tokens past T zero).  (Measured at T = 1, LLaMA-2-7B Q/K/V:
// quantising in every block of the product instead 16.8 us against 14.8, as X
// then queues behind the weights already in flight; counting the codes ready
// so that the product need not wait for this grid's end 16.2 us, as the product
// may then not fetch weights before the previous call has ended.)
// ---------------------------------------------------------------------------
constexpr int kPrepRows = 2, kPrepTokens = 16;

struct Int8PrepArgs {
    const uint16_t* X;
    const uint16_t* B;
    int8_t* xq;
    float* xs;
    __half* R;
    int d, T, tok, r;
};

template <int TOK>
__device__ __forceinline__ void prep_rows(const Int8PrepArgs& a) {
    const int j0 = blockIdx.x * kPrepRows;
    float acc[TOK][kPrepRows] = {};
    for (int i = threadIdx.x; i < a.d / 8; i += kQuantThreads) {
        float w[kPrepRows][8];
#pragma unroll
        for (int j = 0; j < kPrepRows; ++j) {
            const uint4 u = ldg_128(a.B + (int64_t)(j0 + j) * a.d + 8 * i);
            const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 f = __half22float2(u32_as_h2(v[q]));
                w[j][2 * q] = f.x;
                w[j][2 * q + 1] = f.y;
            }
        }
#pragma unroll
        for (int t = 0; t < TOK; ++t) {
            if (t >= a.T) break;
            const uint4 u = ldcg_128(a.X + (int64_t)t * a.d + 8 * i);
            const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 f = __half22float2(u32_as_h2(v[q]));
#pragma unroll
                for (int j = 0; j < kPrepRows; ++j)
                    acc[t][j] = fmaf(f.y, w[j][2 * q + 1], fmaf(f.x, w[j][2 * q], acc[t][j]));
            }
        }
    }
    __shared__ float red[kQuantThreads / 32][TOK * kPrepRows];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int t = 0; t < TOK; ++t) {
        if (t >= a.T) break;
#pragma unroll
        for (int j = 0; j < kPrepRows; ++j) {
            float v = acc[t][j];
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
            if (lane == 0) red[warp][t * kPrepRows + j] = v;
        }
    }
    __syncthreads();
    if ((int)threadIdx.x < min(a.T, TOK) * kPrepRows) {
        float v = 0.f;
        for (int w = 0; w < kQuantThreads / 32; ++w) v += red[w][threadIdx.x];
        a.R[(int64_t)(threadIdx.x / kPrepRows) * a.r + j0 + threadIdx.x % kPrepRows] = __float2half_rn(v);
    }
}

__global__ void __launch_bounds__(kQuantThreads) int8_prep_kernel(const Int8PrepArgs a) {
    pdl_wait();                                  // X is final; the previous call's readers of xq, xs, R are done
    // Only now may the product take its SMs: it fetches weights before it waits
    // itself, and a module's codes may come from a kernel that lets its dependents
    // start early (the token quantiser's codes and scales have a module's format).
    pdl_launch_dependents();
    if ((int)blockIdx.x < a.r / kPrepRows) {
        if (a.T <= 4) prep_rows<4>(a);
        else prep_rows<kPrepTokens>(a);
        return;
    }
    const int t = (int)blockIdx.x - a.r / kPrepRows;
    auto at = [&](int i) {                       // elements 8 i .. + 7 of token t
        return reinterpret_cast<uint2*>(a.xq + ((int64_t)(i >> 3) * a.tok + t) * 64 + (i & 7) * 8);
    };
    if (t < a.T) {
        quantize_token(a.X, t, a.d, a.xs, [&](int i, uint2 q) { *at(i) = q; });
    } else {
        for (int i = threadIdx.x; i < a.d / 8; i += kQuantThreads) *at(i) = make_uint2(0u, 0u);
        if (threadIdx.x == 0) a.xs[t] = 0.f;
    }
}

// ---------------------------------------------------------------------------
// Small T: the product.  Weight streaming; a block's eight warps share a 16-row
// tile of one module, each a share of its k, read as blocks of 16 rows x 128 k
// (2 KB) into a private ring in shared memory with cp.async: a lane copies
// exactly the bytes that it later feeds to the MMA, so no barrier stands
// between copy and use.  mma.m16n8k32 takes k in any order as long as both
// operands agree: lane (g, t) holds the 16 bytes k = 64 h + 16 t .. + 15 of
// rows g and g + 8, and of token g of the staged activations.
// The first blocks of W are in flight while the first launch runs, which has
// waited for everything before the call.
// ---------------------------------------------------------------------------
constexpr int kGemvWarps = 8;
constexpr int kGemvStages = 4;
constexpr int kBlockBytes = 2048;                // 16 rows x 128 k

struct Int8GemvModule {
    const int8_t* q;
    const float* s;
    const __half* A;
    __half* Y;
    int64_t ldY;
    int tile_begin;
};
struct Int8GemvArgs {
    Int8GemvModule mod[GLOWQ_MAX_MODULES];
    const int8_t* xq;       // [d/64][TOK][64]
    const float* xs;        // [TOK]
    const __half* R;        // [T][r]
    int* slots;             // [tile][NT][S][4][32] partial sums (S > 1)
    unsigned int* tickets;  // [tile][NT], zero between calls
    int m, d, T, r, tiles;
    int S;                  // blocks that share a tile's k
    unsigned int* status;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void mma_s8(int c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Shared memory: [codes of X, TOK x k range][rings][R, TOK x r][sums 2 x 8 x NT x 512][token scales][barrier]
struct Int8GemvSmem {
    int ring, rt, red, xs, bar, total;
};
__host__ __device__ inline Int8GemvSmem int8_gemv_smem(int nt, int kblocks, int r) {
    Int8GemvSmem s;
    s.ring = nt * 8 * kblocks * 128;
    s.rt = s.ring + kGemvWarps * kGemvStages * kBlockBytes;
    s.red = (s.rt + nt * 8 * r * 2 + 127) / 128 * 128;
    s.xs = s.red + 2 * kGemvWarps * nt * 512;
    s.bar = s.xs + nt * 8 * 4;
    s.total = s.bar + 16;
    return s;
}

template <int NT>
__global__ void __launch_bounds__(kGemvWarps * 32) int8_gemv_kernel(const __grid_constant__ Int8GemvArgs a) {
    extern __shared__ __align__(128) unsigned char sm[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int ks = blockIdx.x % a.S, tile0 = blockIdx.x / a.S, step = gridDim.x / a.S;
    const int nkb = a.d / 128;
    const int kb0 = (int)((int64_t)ks * nkb / a.S), kb1 = (int)((int64_t)(ks + 1) * nkb / a.S);
    const Int8GemvSmem L = int8_gemv_smem(NT, (nkb + a.S - 1) / a.S, a.r);
    const uint32_t base = smem_u32(sm);
    const uint32_t ring = base + L.ring + warp * kGemvStages * kBlockBytes + lane * 16;
    float* xs = reinterpret_cast<float*>(sm + L.xs);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L.bar);
    const int nsteps = (kb1 - kb0 + kGemvWarps - 1) / kGemvWarps;      // ring blocks per tile (the last may be absent)
    const uint64_t policy = l2_policy_evict_first();
    if (threadIdx.x == 0) {
        mbar_init(bar, 1);
        fence_mbar_init();
    }
    auto module_of = [&](int tile) {
        int mi = 0;
        for (int i = 1; i < a.m; ++i)
            if (tile >= a.mod[i].tile_begin) mi = i;
        return mi;
    };
    // the next block to copy: block pi of tile pt, into ring stage ps
    int pt = tile0, pi = 0, ps = 0;
    const int8_t* psrc = nullptr;                        // row g of the tile, byte 16 t
    auto prefetch = [&]() {
        if (pt < a.tiles) {
            const int kb = kb0 + pi * kGemvWarps + warp;
            if (pi == 0) {
                const Int8GemvModule& md = a.mod[module_of(pt)];
                psrc = md.q + ((int64_t)(pt - md.tile_begin) * 16 + g) * a.d + 16 * t;
            }
            if (kb < kb1) {
                const int8_t* src = psrc + (int64_t)kb * 128;
                const uint32_t dst = ring + ps * kBlockBytes;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    cp_async16(dst + h * 1024, src + h * 64, policy);
                    cp_async16(dst + h * 1024 + 512, src + h * 64 + (int64_t)8 * a.d, policy);
                }
            }
            if (++pi == nsteps) {
                pi = 0;
                pt += step;
            }
        }
        if (++ps == kGemvStages) ps = 0;
        cp_async_commit();                               // one group per call, empty ones too: waits count groups
    };
    // A fragments of columns j0 .. j0 + 63: lane (g, t) holds columns j0 + 16 t .. + 15 of rows g ([0], [1]) and
    // g + 8 ([2], [3]), the MMA's k in the order that the reads of R use too
    auto load_a = [&](int tile, int j0, uint4 (&f)[4]) {
        const Int8GemvModule& md = a.mod[module_of(tile)];
        const __half* A = md.A + ((int64_t)(tile - md.tile_begin) * 16 + g) * a.r + j0 + 16 * t;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            f[p] = f[2 + p] = make_uint4(0, 0, 0, 0);
            if (j0 + 16 * t + 8 * p < a.r) {
                f[p] = ldg_stream(A + 8 * p);
                f[2 + p] = ldg_stream(A + 8 * p + (int64_t)8 * a.r);
            }
        }
    };
    for (int i = 0; i < kGemvStages - 1; ++i) prefetch();
    __syncthreads();                                     // the barrier is initialised
    pdl_wait();                                          // codes, scales and R of this call are complete
    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        const uint32_t bytes = (uint32_t)(NT * 8 * 128) * (uint32_t)(kb1 - kb0);
        mbar_arrive_expect_tx(bar, bytes);
        bulk_g2s(base, a.xq + (int64_t)kb0 * (NT * 8 * 128), bytes, bar);
    }
    for (int i = threadIdx.x; i < NT * a.r; i += kGemvWarps * 32) {   // 8 halves each
        *reinterpret_cast<uint4*>(sm + L.rt + i * 16) = ldcg_128_if(a.R + i * 8, i * 8 / a.r < a.T);
    }
    if (threadIdx.x < NT * 8) xs[threadIdx.x] = ldcg_f32(a.xs + threadIdx.x);
    mbar_wait(bar, 0, a.status);
    __syncthreads();
    int cs = 0, par = 0;
    for (int tile = tile0; tile < a.tiles; tile += step, par ^= 1) {
        int acc[NT][4] = {};
        // the tile's first 64 columns of A, loaded ahead by the warps that will apply them
        uint4 af[4];
        const int mi = module_of(tile);
        const bool corrects = a.r > 0 && warp < NT && a.mod[mi].A;
        if (corrects) load_a(tile, 0, af);
        for (int i = 0; i < nsteps; ++i) {
            prefetch();
            cp_async_wait<kGemvStages - 1>();
            const int kb = i * kGemvWarps + warp;        // within this block's k range
            if (kb0 + kb < kb1) {
                const unsigned char* src = sm + L.ring + (warp * kGemvStages + cs) * kBlockBytes + lane * 16;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint4 lo = *reinterpret_cast<const uint4*>(src + h * 1024);
                    const uint4 hi = *reinterpret_cast<const uint4*>(src + h * 1024 + 512);
                    const unsigned char* xp = sm + (kb * 2 + h) * (NT * 8 * 64) + g * 64 + t * 16;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint4 x = *reinterpret_cast<const uint4*>(xp + n * 512);
                        mma_s8(acc[n], lo.x, hi.x, lo.y, hi.y, x.x, x.y);
                        mma_s8(acc[n], lo.z, hi.z, lo.w, hi.w, x.z, x.w);
                    }
                }
            }
            if (++cs == kGemvStages) cs = 0;
        }
        // the warps' sums meet in shared memory (double buffered: one barrier per tile)
        int4* red = reinterpret_cast<int4*>(sm + L.red + par * kGemvWarps * NT * 512);
#pragma unroll
        for (int n = 0; n < NT; ++n) red[(warp * NT + n) * 32 + lane] = make_int4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
        __syncthreads();
        if (warp >= NT) continue;                        // warp n finishes tokens 8 n .. 8 n + 7
        const int n = warp;
        const Int8GemvModule& md = a.mod[mi];
        const int row0 = (tile - md.tile_begin) * 16;
        int v[4] = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kGemvWarps; ++w) {
            const int4 p = red[(w * NT + n) * 32 + lane];
            v[0] += p.x, v[1] += p.y, v[2] += p.z, v[3] += p.w;
        }
        if (a.S > 1) {
            // this block's share of k to its slot; the share that counts last adds them all (integers: any order)
            int* slot = a.slots + (((int64_t)tile * NT + n) * a.S) * 128 + lane;
#pragma unroll
            for (int q = 0; q < 4; ++q) __stcg(slot + ks * 128 + q * 32, v[q]);
            __threadfence();
            __syncwarp();
            unsigned int prev = 0;
            unsigned int* tk = a.tickets + tile * NT + n;
            if (lane == 0)
                asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(prev) : "l"(tk) : "memory");
            prev = __shfl_sync(~0u, prev, 0);
            if (prev != (unsigned)(a.S - 1)) continue;
            if (lane == 0) atomicExch(tk, 0u);           // every share has counted: ready for the next call
            __threadfence();
            for (int s = 0; s < a.S; ++s) {
                if (s == ks) continue;
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] += __ldcg(slot + s * 128 + q * 32);
            }
        }
        float c[4] = {0.f, 0.f, 0.f, 0.f};
        if (corrects) {
            for (int j0 = 0; j0 < a.r; j0 += 64) {
                if (j0 > 0) load_a(tile, j0, af);
                uint4 x[2];
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const int j = j0 + 16 * t + 8 * p;
                    x[p] = make_uint4(0, 0, 0, 0);
                    if (j < a.r) x[p] = *reinterpret_cast<const uint4*>(sm + L.rt + ((n * 8 + g) * a.r + j) * 2);
                }
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const uint32_t a1[4] = {af[p].x, af[2 + p].x, af[p].y, af[2 + p].y}, b1[2] = {x[p].x, x[p].y};
                    const uint32_t a2[4] = {af[p].z, af[2 + p].z, af[p].w, af[2 + p].w}, b2[2] = {x[p].z, x[p].w};
                    mma_16816(c, a1, b1);
                    mma_16816(c, a2, b2);
                }
            }
        }
        const float s0 = __ldg(md.s + row0 + g), s1 = __ldg(md.s + row0 + g + 8);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int tok = n * 8 + 2 * t + e;
            if (tok < a.T) {
                const float st = xs[tok];
                __half* y = md.Y + (int64_t)tok * md.ldY + row0 + g;
                y[0] = __float2half_rn(fmaf((float)v[e] * st, s0, c[e]));
                y[8] = __float2half_rn(fmaf((float)v[2 + e] * st, s1, c[2 + e]));
            }
        }
    }
    cp_async_wait<0>();
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
cudaError_t launch_pack_int8(const float* W, int64_t O, int64_t d, int8_t* codes, float* scales, cudaStream_t st) {
    pack_int8_kernel<<<(unsigned)O, kQuantThreads, 0, st>>>(W, d, codes, scales);
    return cudaGetLastError();
}
cudaError_t launch_dequant_int8(const int8_t* codes, const float* scales, int64_t O, int64_t d, uint16_t* out,
                                cudaStream_t st) {
    dequant_int8_kernel<<<(unsigned)O, 256, 0, st>>>(codes, scales, d, reinterpret_cast<__half*>(out));
    return cudaGetLastError();
}
cudaError_t launch_pdl(const void* fn, unsigned grid, unsigned block, size_t smem, cudaStream_t st, void** args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, fn, args);
}
cudaError_t launch_quantize_act_int8(const uint16_t* X, int64_t T, int64_t d, int8_t* codes, float* scales,
                                     cudaStream_t st) {
    void* args[] = {(void*)&X, (void*)&d, (void*)&codes, (void*)&scales};
    return launch_pdl((const void*)quantize_act_int8_kernel, (unsigned)T, kQuantThreads, 0, st, args);
}

cudaError_t launch_quantize_beside(const uint16_t* X, int64_t T, int64_t d, int8_t* codes, float* scales,
                                   unsigned int* ready, bool first, cudaStream_t st) {
    void* args[] = {(void*)&X, (void*)&d, (void*)&codes, (void*)&scales, (void*)&ready, (void*)&first};
    return launch_pdl((const void*)int8_quantize_kernel, (unsigned)T, kQuantThreads, 0, st, args);
}

// Token width (a multiple of 8) of the small-T kernels.
int int8_small_tokens(int64_t T) { return T <= 8 ? 8 : 16; }

// Decomposition of the small-T product: the fewest shares of k that leave two
// blocks an SM (or one, if the staged activations need the room) and a tile or
// more for each, or whose shares are down to two blocks per warp.
Int8GemvPlan plan_int8_gemv(int64_t T, int64_t d, int64_t tiles, int r, int num_sms) {
    Int8GemvPlan p;
    const int nt = int8_small_tokens(T) / 8, nkb = (int)(d / 128);
    for (p.S = 1; p.S < nkb; ++p.S) {
        if (int8_gemv_smem(nt, (nkb + p.S - 1) / p.S, r).total > 227 * 1024) continue;
        if (tiles * p.S >= num_sms || (nkb + p.S) / (p.S + 1) < 2 * kGemvWarps) break;
    }
    p.smem = int8_gemv_smem(nt, (nkb + p.S - 1) / p.S, r).total;
    p.ok = p.smem <= 227 * 1024 && (p.S == 1 || tiles * nt <= kInt8MaxTickets) && tiles < (1 << 24);
    const int64_t slots = (int64_t)num_sms * (p.smem <= 113 * 1024 ? 2 : 1) / p.S;
    p.grid = (int)(tiles < slots ? tiles : (slots < 1 ? 1 : slots)) * p.S;
    p.slot_bytes = p.S > 1 ? (size_t)tiles * nt * p.S * 512 : 0;
    return p;
}

template <int NT>
static cudaError_t launch_int8_gemv_t(const Int8GemvArgs& a, const Int8GemvPlan& p, cudaStream_t st) {
    const void* fn = (const void*)int8_gemv_kernel<NT>;
    static SmemLimit limit;
    cudaError_t e = limit.raise(fn, 227 * 1024);
    if (e != cudaSuccess) return e;
    void* args[] = {(void*)&a};
    return launch_pdl(fn, (unsigned)p.grid, kGemvWarps * 32, (size_t)p.smem, st, args);
}

cudaError_t launch_int8_small(const Int8ModuleView* mods, int m, int d, int T, int r, const uint16_t* X,
                              const uint16_t* B, uint16_t* R, int8_t* xq, float* xs, unsigned int* tickets, int* slots,
                              const Int8GemvPlan& p, cudaStream_t st) {
    const int tok = int8_small_tokens(T);
    Int8PrepArgs pa = {X, B, xq, xs, reinterpret_cast<__half*>(R), d, T, tok, r};
    void* pargs[] = {(void*)&pa};
    cudaError_t e = launch_pdl((const void*)int8_prep_kernel, (unsigned)(r / kPrepRows + tok), kQuantThreads, 0, st, pargs);
    if (e != cudaSuccess) return e;
    Int8GemvArgs a = {};
    int tile = 0;
    for (int i = 0; i < m; ++i) {
        a.mod[i] = {mods[i].q, mods[i].s, reinterpret_cast<const __half*>(mods[i].A), reinterpret_cast<__half*>(mods[i].Y),
                    mods[i].ldY, tile};
        tile += (int)(mods[i].O / 16);
    }
    a.xq = xq;
    a.xs = xs;
    a.R = reinterpret_cast<const __half*>(R);
    a.slots = slots;
    a.tickets = tickets;
    a.m = m;
    a.d = d;
    a.T = T;
    a.r = r;
    a.tiles = tile;
    a.S = p.S;
    a.status = device_status_ptr();
    return T <= 8 ? launch_int8_gemv_t<1>(a, p, st) : launch_int8_gemv_t<2>(a, p, st);
}

}  // namespace glowq
