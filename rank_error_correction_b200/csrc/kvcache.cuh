// kvcache.cuh -- device views of the paged 8-bit key/value cache and of a
// step's batch (layouts in glowq.h).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "glowq.h"

namespace glowq {

constexpr int kKvPage = GLOWQ_KV_PAGE;
constexpr int kKvReadMax = 1 << 29;      // tokens of a read, and its first position, at most

struct KvCacheView {
    int8_t* k_codes;     // [pages][kv_heads][D/64][64 tokens][64]
    int8_t* v_codes;     // [pages][kv_heads][D][64 tokens]
    float* k_scales;     // [pages][kv_heads]
    float* v_scales;
    uint16_t* k_tail;    // [slots][kv_heads][64 tokens][D]
    uint16_t* v_tail;
    int64_t pages, slots;
    int kv_heads, head_dim;
};
struct KvBatchView {
    const int *q_start, *kv_len, *table, *slot;
    int n_seq, max_pages, T, max_new;
};

// Pages that n consecutive tokens may touch.
__host__ __device__ inline int kv_touched_pages(int n) { return n <= 0 ? 0 : (int)(((int64_t)n + 2 * kKvPage - 2) / kKvPage); }

// Sequence b of the batch: rows [q0, q0 + nq) of the step, cached length len
// after it, the first row's position.  ok: the rows are inside the batch.
struct KvSeq {
    int q0, nq, len, start, slot;
    bool ok;
};
__device__ __forceinline__ KvSeq kv_sequence(const KvBatchView& b, int i) {
    KvSeq s;
    s.q0 = ldcg_s32(b.q_start + i);
    const int q1 = ldcg_s32(b.q_start + i + 1);
    s.len = ldcg_s32(b.kv_len + i);
    s.slot = ldcg_s32(b.slot + i);
    s.ok = s.q0 >= 0 && q1 >= s.q0 && q1 <= b.T && q1 - s.q0 <= b.max_new && s.len >= 0;
    s.nq = s.ok ? q1 - s.q0 : 0;
    s.start = s.ok ? s.len - s.nq : 0;
    return s;
}

cudaError_t launch_kv_append(const KvCacheView& c, const KvBatchView& b, const uint16_t* Q, int64_t ldQ, int q_heads,
                             const uint16_t* K, int64_t ldK, const uint16_t* V, int64_t ldV, const float* rope,
                             int rope_len, uint16_t* Q_out, int64_t ldQo, cudaStream_t st);
cudaError_t launch_kv_read(const KvCacheView& c, const KvBatchView& b, const int* first, int count, uint16_t* K,
                           uint16_t* V, cudaStream_t st);

// A row whose scores are all -infinity (an infinite query, say) has no softmax
// and becomes NaN, unlike one that sees nothing, which is zero: to tell them
// apart, a row that sees something takes this as its maximum.
constexpr float kLeastScore = -3e38f;

// attention.cu
struct KvAttnPlan {
    bool tc;             // many rows: attention_tc.cu
    int rows;            // query rows of a block at a time: 8 or 16
    int blocks, sms;
    int S;               // tc: shares of a unit's tokens
    size_t partial_bytes;
};
KvAttnPlan plan_kv_attention(const KvBatchView& b, int G, int kv_heads, int head_dim, int num_sms);
cudaError_t launch_kv_attention(const KvCacheView& c, const KvBatchView& b, const uint16_t* Q, int64_t ldQ, int q_heads,
                                float scale, uint16_t* Y, int64_t ldY, unsigned int* tickets, float* partial,
                                const KvAttnPlan& p, cudaStream_t st);

// attention_tc.cu: many rows on the tensor cores
struct KvTcShares {
    int S;               // of a unit's tokens
    double us;           // expected
};
KvTcShares kv_tc_shares(const KvBatchView& b, int G, int kv_heads, int num_sms);
size_t kv_tc_partial_bytes(const KvBatchView& b, int G, int kv_heads, int S, int head_dim);
cudaError_t launch_kv_attention_tc(const KvCacheView& c, const KvBatchView& b, const uint16_t* Q, int64_t ldQ, int q_heads,
                                   float scale, uint16_t* Y, int64_t ldY, unsigned int* tickets, float* partial, int S,
                                   cudaStream_t st);

}  // namespace glowq
