// Kernel launchers behind the C ABI. Each validates nothing (the ABI layer has
// already checked every argument) and returns the hipError_t of its launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "q4.h"
#include "validate.h"

namespace q4k {

// Block format of a weight stream.
enum class WeightFormat { kQ4_0, kQ8_0 };

hipError_t launch_dequant(WeightFormat fmt, const uint8_t *w, size_t n_blocks, float *out,
                          hipStream_t s);
hipError_t launch_gemv(WeightFormat fmt, const float *a, const uint8_t *w, float *y, int M, int N,
                       int K, hipStream_t s);
// a: [M, K] bfloat16 bit patterns, 1 <= M <= 8.
hipError_t launch_gemv_bf16(WeightFormat fmt, const uint16_t *a, const uint8_t *w, float *y, int M,
                            int N, int K, hipStream_t s);
// Prepared activations for the GEMV: launch_gemv_prepare writes
// q4v::gemv_prepare_bytes(M, K) bytes of operands for the format; the
// prepared GEMV reads them instead of `a` (K % 256 == 0 only).
hipError_t launch_gemv_prepare(WeightFormat fmt, const float *a, void *prep, int M, int K,
                               hipStream_t s);
hipError_t launch_gemv_prepared(WeightFormat fmt, const void *prep, const uint8_t *w, float *y,
                                int M, int N, int K, hipStream_t s);
// a_q: the [M, K/32] Q8_0 block stream of the activations, 1 <= M <= 8.
hipError_t launch_gemv_q8a(WeightFormat fmt, const uint8_t *a_q, const uint8_t *w, float *y, int M,
                           int N, int K, hipStream_t s);
// K split across workgroups: partials of sp.splits splits into `workspace`
// (sp.splits * M * N f32), then summed into y in split order. sp.splits <= 1
// runs launch_gemv's kernel (workspace unused).
hipError_t launch_gemv_splitk(WeightFormat fmt, const float *a, const uint8_t *w, float *y, int M,
                              int N, int K, const q4v::GemvSplit &sp, void *workspace,
                              hipStream_t s);
// workspace: q4v::gemm_workspace_bytes(M, N, K) bytes (always used: the row
// exponents, then on the split path the two-term operands).
hipError_t launch_gemm(WeightFormat fmt, const float *a, const uint8_t *w, float *y, int M, int N,
                       int K, void *workspace, hipStream_t s);
// The same without a workspace: the library's own device scratch of
// kGemmScratchBytes per GPU, rows taken in chunks that fit it. Calls that
// overlap in time on one GPU race on the scratch.
constexpr size_t kGemmScratchBytes = Q4_GEMM_SCRATCH_BYTES;
hipError_t launch_gemm_noalloc(WeightFormat fmt, const float *a, const uint8_t *w, float *y, int M,
                               int N, int K, hipStream_t s);
// a: [M, K] bfloat16 bit patterns. workspace:
// q4v::gemm_bf16_workspace_bytes(M, N, K) bytes (always used).
hipError_t launch_gemm_bf16(WeightFormat fmt, const uint16_t *a, const uint8_t *w, float *y, int M,
                            int N, int K, void *workspace, hipStream_t s);
// a_q: the [M, K/32] Q8_0 block stream of the activations. workspace:
// q4v::gemm_q8a_workspace_bytes(M, N, K) bytes (always used).
hipError_t launch_gemm_q8a(WeightFormat fmt, const uint8_t *a_q, const uint8_t *w, float *y, int M,
                           int N, int K, void *workspace, hipStream_t s);
hipError_t launch_q8_quantize(const float *x, size_t n_blocks, uint8_t *out, hipStream_t s);
hipError_t launch_q4_quantize(const float *x, size_t n_blocks, uint8_t *out, hipStream_t s);

// E4M3 codes with one scale per 128 columns of a row (block_rows 1) or per
// 128 x 128 tile (128).
hipError_t launch_f8_quantize(const float *x, uint8_t *q, float *s, int M, int K, int block_rows,
                              hipStream_t st);
hipError_t launch_f8_quantize_bf16(const uint16_t *x, uint8_t *q, float *s, int M, int K,
                                   int block_rows, hipStream_t st);
hipError_t launch_f8_dequant(const uint8_t *q, const float *s, float *out, int M, int K,
                             int block_rows, hipStream_t st);
// y: [M, N] bfloat16. K <= 2^22.
hipError_t launch_f8_gemm(const uint8_t *a, const float *a_s, const uint8_t *w, const float *w_s,
                          uint16_t *y, int M, int N, int K, hipStream_t st);
// The router. workspace: q4v::route_workspace_bytes(T, E, top_k) bytes.
hipError_t launch_route(const float *logits, int *ids, float *weights, int *offsets, int *order,
                        void *workspace, int T, int E, int top_k, bool renorm, hipStream_t st);
// The router with scores, a bias and groups of experts; the same workspace.
struct RouteGroups {
    const float *bias;   // [E], or null
    bool sigmoid, renorm;
    int n_groups, top_groups, group_best;
    float scale;
};
hipError_t launch_route_groups(const float *logits, const RouteGroups &g, int *ids, float *weights,
                               int *offsets, int *order, void *workspace, int T, int E, int top_k,
                               hipStream_t st);
// A row of results in the form that the next product reads.
enum class RowForm { kF32, kBf16, kQ8_0, kE4M3 };
struct RowOut {
    void *y;    // values, blocks or codes
    float *s;   // E4M3: the scales
};
// The norm of the residual stream. x, residual, sum and dense in f32 or bfloat16
// (bf16); weights, residual, sum and dense may be null, sum may be residual.
struct NormArgs {
    const void *x;
    const float *weights;
    int share;
    const void *residual;
    void *sum;
    const float *gamma;
    float eps;
    void *dense;
    RowOut out;
    int M, K;
};
hipError_t launch_norm(bool bf16, RowForm form, const NormArgs &a, hipStream_t st);
// The gated activation. gate and up in f32 or bfloat16, rows ld elements apart; up
// may be null.
struct ActArgs {
    const void *gate, *up;
    int ld, act;
    RowOut out;
    int M, K;
};
hipError_t launch_act(bool bf16, RowForm form, const ActArgs &a, hipStream_t st);
// The grouped products over Q4_0 and Q8_0 weights: f32 or bfloat16 (bf16)
// activations; order may be null. workspace: q4v::grouped_workspace_bytes.
hipError_t launch_gemm_grouped(WeightFormat fmt, bool bf16, const void *a, const uint8_t *w,
                               const int *offsets, const int *order, int share, float *y, int G,
                               int M, int N, int K, void *workspace, hipStream_t st);
// order may be null; the activations' codes span less than 2^31 bytes.
hipError_t launch_f8_gemm_grouped(const uint8_t *a, const float *a_s, const uint8_t *w,
                                  const float *w_s, const int *offsets, const int *order, int share,
                                  uint16_t *y, int G, int M, int N, int K, hipStream_t st);

}  // namespace q4k
