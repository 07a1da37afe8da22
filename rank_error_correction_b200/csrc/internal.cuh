// internal.cuh -- declarations shared by the translation units of libglowq.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "glowq.h"

namespace glowq {

// Host-side view of one module of a group (validated by api.cu).
struct ModuleView {
    const uint32_t* q;   // packed 4-bit codes [O][d/8]
    const void* s;       // INT4: fp16 scales [O][d/128]; MXFP4 / NVFP4: scale bytes
    const uint8_t* z;    // INT4 zeros (nullptr for FP4)
    const float* ts;     // NVFP4 tensor scale (device), else nullptr
    const uint16_t* A;   // nullptr: correction off for this module
    uint16_t* Y;
    int64_t ldY;
    int64_t O;
};

constexpr int kDecodeMaxTokens = 16;
// Tokens up to which the tcgen05 path uses 64-token pair tiles and may split k.
constexpr int kSmallBatchMaxTokens = 64;

// Workspace layout: [zero region][R partials][solo R][k-split slots].  The
// zero region holds the decode hand-off flags (bytes 0..255) and the k-split
// tickets (bytes 256..4095, one u32 per CTA of a split tile); it must be zero
// before a call and every call that completes leaves it zero.
constexpr size_t kWorkspaceZeroBytes = 4096;
constexpr size_t kTicketOffsetBytes = 256;
constexpr int kMaxTickets = (int)((kWorkspaceZeroBytes - kTicketOffsetBytes) / 4);
constexpr int kMaxSplit = 8;          // parts per tile
constexpr int kMinSplitBlocks = 8;    // k-blocks (of 64) per part, at least
// Costs of the small-batch work decomposition in k-blocks of streamed weights
// (fitted to a sweep of S = 1..8 over the LLaMA-2-7B / LLaMA-3.1-8B /
// LLaMA-2-13B units at T = 32 and 64 on B200, ~0.37 us per k-block): a work
// unit's fixed cost (ring fill, accumulator drain, stores), and a split tile's
// partial-sum traffic and reduction, a base plus a share per part.
constexpr int kUnitCost = 15;
constexpr int kSplitBaseCost = 6;
constexpr int kSplitPartCost = 3;

// Argument checks of glowq_solo_forward, without the workspace (api.cu).
glowq_status validate_solo_call(const glowq_module* mod, int64_t d, const uint16_t* B, int32_t r, const uint16_t* X,
                                int64_t T);

// Device address of this device's status word (bounded-wait timeouts).
unsigned int* device_status_ptr();

// decode.cu
// Corrected GEMV over the stacked rows (T <= 16), one launch.  With r > 0 it
// also computes R = X B^T (written to R) from fp32 partial sums in `partial`
// (decode_partial_bytes(T, r)); `flags` are the first 256 bytes of the
// workspace's zero region, which every completed call leaves zero.
cudaError_t launch_gemv_decode(const ModuleView* mods, int m, int d, int T, int r, const uint16_t* X,
                               const uint16_t* B, uint16_t* R, unsigned int* flags, float* partial, int num_sms,
                               cudaStream_t st, int fmt = GLOWQ_FMT_INT4, const float* tok_scale = nullptr);
size_t decode_partial_bytes(int64_t T, int r);
// pack.cu
cudaError_t launch_pack_int4(const float* W, int64_t O, int64_t d, uint32_t* q, uint16_t* s, uint8_t* z,
                             cudaStream_t st);
cudaError_t launch_dequant_int4(const uint32_t* q, const uint16_t* s, const uint8_t* z, int64_t O, int64_t d,
                                uint16_t* out, cudaStream_t st);
cudaError_t launch_error_norms(const float* W, const uint32_t* q, const uint16_t* s, const uint8_t* z,
                               int64_t O, int64_t d, double* out_rows, cudaStream_t st);
// fp4.cu
cudaError_t launch_quantize_act_e4m3(const uint16_t* X, int64_t T, int64_t d, uint8_t* codes, float* scales,
                                     uint16_t* Xq, cudaStream_t st);
cudaError_t launch_pack_fp4(int fmt, const float* W, int64_t O, int64_t d, uint32_t* codes, uint8_t* scales,
                            float* tensor_scale, cudaStream_t st);
cudaError_t launch_dequant_fp4(int fmt, const uint32_t* codes, const uint8_t* scales, const float* tensor_scale,
                               int64_t O, int64_t d, uint16_t* out, cudaStream_t st);
// A launch that may begin while the preceding kernel of the stream ends (the
// kernel waits for it with pdl_wait before it touches anything it wrote).
// A kernel's limit of dynamic shared memory, raised once per device: the call
// takes 2.4 us of the host, as much as a launch.  One object for each kernel.
class SmemLimit {
    std::atomic<uint64_t> raised_{0};

public:
    cudaError_t raise(const void* fn, int bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 64 && (raised_.load(std::memory_order_acquire) >> dev & 1)) return cudaSuccess;
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess && dev < 64) raised_.fetch_or((uint64_t)1 << dev, std::memory_order_release);
        return e;
    }
};
cudaError_t launch_pdl(const void* fn, unsigned grid, unsigned block, size_t smem, cudaStream_t st, void** args);

// int8.cu: 8-bit integer weights and activations
struct Int8ModuleView {
    const int8_t* q;     // codes [O][d]
    const float* s;      // scales [O]
    const uint16_t* A;   // nullptr: correction off for this module
    uint16_t* Y;
    int64_t ldY;
    int64_t O;
};
constexpr int64_t kInt8MaxD = 131072;          // 127^2 d < 2^31
constexpr int kInt8SmallTokens = 16;           // tokens up to which the weight-streaming product runs
constexpr int kInt8ZeroBytes = 65536;          // tickets at the workspace's start
constexpr int kInt8MaxTickets = kInt8ZeroBytes / 4 - 64;
// Behind the tickets, two counters between the quantiser and the product that
// runs beside its end: tokens quantised so far, blocks of the product done with
// waiting (the last one returns both to zero).
constexpr int kInt8Ready = kInt8MaxTickets, kInt8Done = kInt8MaxTickets + 1;
// Decomposition of the small-T product: S blocks share a tile's k.
struct Int8GemvPlan {
    bool ok;             // false: the shape is left to the tensor-core GEMM
    int S, grid, smem;
    size_t slot_bytes;   // partial sums (S > 1)
};
int int8_small_tokens(int64_t T);
Int8GemvPlan plan_int8_gemv(int64_t T, int64_t d, int64_t tiles, int r, int num_sms);
cudaError_t launch_pack_int8(const float* W, int64_t O, int64_t d, int8_t* codes, float* scales, cudaStream_t st);
cudaError_t launch_dequant_int8(const int8_t* codes, const float* scales, int64_t O, int64_t d, uint16_t* out,
                                cudaStream_t st);
cudaError_t launch_quantize_act_int8(const uint16_t* X, int64_t T, int64_t d, int8_t* codes, float* scales,
                                     cudaStream_t st);
cudaError_t launch_int8_small(const Int8ModuleView* mods, int m, int d, int T, int r, const uint16_t* X,
                              const uint16_t* B, uint16_t* R, int8_t* xq, float* xs, unsigned int* tickets, int* slots,
                              const Int8GemvPlan& p, cudaStream_t st);
// The token quantiser behind a kernel of the same call that has waited for X: its end implies that kernel's.
// It counts the tokens that are done on `ready`.
cudaError_t launch_quantize_beside(const uint16_t* X, int64_t T, int64_t d, int8_t* codes, float* scales,
                                   unsigned int* ready, bool first, cudaStream_t st);
// int8_gemm.cu: T > 16 on the tensor cores.  `rounds` whole tiles per pair
// (tiles [0, whole)), then the other tiles' k-blocks as one run of `blocks` cut
// evenly among the first `sharers` pairs (every one has a share, in at most
// `segments` tiles).
struct I8Split {
    int pairs, rounds, nkb, sharers, segments;
    int64_t whole;
    int blocks;          // below pairs nkb, so that blocks x pairs fits an int
};
// Where a pair's share begins (at `sharers` and behind: the end of the run).
__host__ __device__ inline int i8_share(const I8Split& s, int pair) {
    return pair >= s.sharers ? s.blocks : (int)((unsigned)s.blocks * (unsigned)pair / (unsigned)s.sharers);
}
struct I8GemmPlan {
    int bn;              // tokens per pair tile
    I8Split split;
    int64_t rest;        // split tiles
    size_t slot_bytes;   // their partial sums
};
I8GemmPlan plan_int8_gemm(int64_t T, int64_t d, int64_t mtiles, int num_sms);
cudaError_t launch_int8_project(const uint16_t* X, const uint16_t* B, int64_t T, int d, int r, uint16_t* R,
                                cudaStream_t st);
cudaError_t launch_int8_gemm(const Int8ModuleView* mods, int m, int d, int64_t T, int r, const int8_t* xq,
                             const float* xs, const uint16_t* R, unsigned int* tickets, int* slots, const I8GemmPlan& p,
                             cudaStream_t st);
// solve.cu: the offline group solve (float64)
struct SolveModule {
    const float* W;      // O x d fp32 weights
    const uint32_t* q;   // INT4 packed codes
    const uint16_t* s;   // fp16 scales
    const uint8_t* z;    // zeros
    int64_t O;
};
size_t solve_workspace_bytes(int64_t M, int64_t d, int l);
glowq_status group_solve_impl(const SolveModule* mods, int m, int64_t d, const double* Sh, const double* Shp,
                              int r, int p, int qit, const double* Omega, double* A, double* B, double* sing,
                              double* gec, uint16_t* A16, uint16_t* B16, void* workspace, unsigned int* err,
                              cudaStream_t st);
// prefill.cu: TMA tensor maps (driver entry point resolved at run time)
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn();
// 2-D row-major tensor [outer][inner], row pitch `pitch` bytes, box {box_inner, box_outer}.
bool make_map(CUtensorMap* map, CUtensorMapDataType dt, const void* base, uint64_t inner, uint64_t outer,
              uint64_t pitch, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle sw);
// `partial`: scratch of prefill_partial_bytes(T, r) for the split R projection
// (nullptr: one slice of d per CTA, R written directly).
// `tickets` (zeroed workspace words) and `slots` (max_slots fp32 partial
// tiles of prefill_slot_bytes) enable the k-split; nullptr / 0: whole tiles.
glowq_status prefill_group_forward(const ModuleView* mods, int m, int d, const uint16_t* B, int r,
                                   const uint16_t* X, int64_t T, uint16_t* R, float* partial, int num_sms,
                                   cudaStream_t st, int fmt = GLOWQ_FMT_INT4, const float* tok_scale = nullptr,
                                   uint16_t* R_scaled = nullptr, unsigned int* tickets = nullptr,
                                   float* slots = nullptr, int64_t max_slots = 0);
size_t prefill_partial_bytes(int64_t T, int r);
// Work decomposition of the tcgen05 GEMM: token width bn of the pair tiles,
// tiles [0, split_from) whole, the rest split into S parts of kbs k-blocks;
// slots = fp32 partial tiles the split needs.
struct SplitPlan {
    int bn;
    int64_t ntiles_n, ntiles, split_from;
    int S, kbs;
    int64_t slots;
};
SplitPlan plan_prefill_split(int64_t T, int d, int64_t mtiles, int pairs, int64_t max_slots);
int gemm_max_pairs(int num_sms);
int prefill_tile_n(int64_t T);
size_t prefill_slot_bytes(int bn);

}  // namespace glowq
