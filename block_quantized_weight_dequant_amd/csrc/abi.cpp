// The exported C ABI (include/q4.h, include/f8.h): validate every argument,
// then enqueue the kernel on the caller's stream. Only the functions declared
// there are exported from the shared library (it is built with hidden
// visibility).
#include "f8.h"
#include "q4.h"

#include "launch.h"
#include "validate.h"

#define Q4_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

int launched(hipError_t e) { return e == hipSuccess ? Q4_OK : Q4_ERR_LAUNCH; }

hipStream_t as_stream(void *s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace

Q4_EXPORT int q4_abi_version(void) { return Q4_ABI_VERSION; }

Q4_EXPORT const char *q4_status_string(int status)
{
    switch (status) {
    case Q4_OK: return "ok";
    case Q4_ERR_NULL: return "a required pointer is NULL";
    case Q4_ERR_SHAPE: return "invalid shape (K must be a positive multiple of 32, sizes non-negative, "
                              "element counts a multiple of 32, GEMV rows in [0, 8])";
    case Q4_ERR_SIZE: return "a byte or element count does not match the shape";
    case Q4_ERR_ALIGN: return "a pointer is not 16-byte aligned";
    case Q4_ERR_ALIAS: return "an output overlaps an input";
    case Q4_ERR_LAUNCH: return "the HIP runtime refused the kernel launch";
    case Q4_ERR_WORKSPACE: return "the workspace is smaller than the GEMM's workspace_bytes function asks";
    default: return "unknown status";
    }
}

// Shared bodies of the Q4_0 and Q8_0 entry points.
static int dequant(q4k::WeightFormat fmt, size_t block_bytes, const void *w_q, size_t w_bytes,
                   float *out, size_t out_elems, void *stream)
{
    bool empty = false;
    int st = q4v::check_dequant(w_q, w_bytes, out, out_elems, block_bytes, &empty);
    if (st != Q4_OK || empty)
        return st;
    return launched(q4k::launch_dequant(fmt, static_cast<const uint8_t *>(w_q), w_bytes / block_bytes,
                                        out, as_stream(stream)));
}

static int gemv(q4k::WeightFormat fmt, size_t block_bytes, const float *a, const void *w_q,
                size_t w_bytes, float *y, int M, int N, int K, void *stream)
{
    bool empty = false;
    int st = q4v::check_product(a, sizeof(float), w_q, w_bytes, y, M, N, K, Q4_GEMV_MAX_ROWS,
                                block_bytes, &empty);
    if (st != Q4_OK || empty)
        return st;
    return launched(q4k::launch_gemv(fmt, a, static_cast<const uint8_t *>(w_q), y, M, N, K,
                                     as_stream(stream)));
}

static int gemm(q4k::WeightFormat fmt, size_t block_bytes, const float *a, const void *w_q,
                size_t w_bytes, float *y, int M, int N, int K, void *workspace,
                size_t workspace_bytes, void *stream)
{
    bool empty = false;
    int st = q4v::check_product(a, sizeof(float), w_q, w_bytes, y, M, N, K, 0, block_bytes, &empty);
    if (st != Q4_OK || empty)
        return st;
    st = q4v::check_workspace(q4v::gemm_workspace_bytes(M, N, K), a, sizeof(float), w_q, w_bytes,
                              y, M, N, K, workspace, workspace_bytes);
    if (st != Q4_OK)
        return st;
    return launched(q4k::launch_gemm(fmt, a, static_cast<const uint8_t *>(w_q), y, M, N, K,
                                     workspace, as_stream(stream)));
}

static int gemm_noalloc(q4k::WeightFormat fmt, size_t block_bytes, const float *a, const void *w_q,
                        size_t w_bytes, float *y, int M, int N, int K, void *stream)
{
    bool empty = false;
    int st = q4v::check_product(a, sizeof(float), w_q, w_bytes, y, M, N, K, 0, block_bytes, &empty);
    if (st != Q4_OK || empty)
        return st;
    return launched(q4k::launch_gemm_noalloc(fmt, a, static_cast<const uint8_t *>(w_q), y, M, N, K,
                                             as_stream(stream)));
}

static int gemv_splitk(q4k::WeightFormat fmt, size_t block_bytes, const float *a, const void *w_q,
                       size_t w_bytes, float *y, int M, int N, int K, int splits, void *workspace,
                       size_t workspace_bytes, void *stream)
{
    bool empty = false;
    int st = q4v::check_product(a, sizeof(float), w_q, w_bytes, y, M, N, K, Q4_GEMV_MAX_ROWS,
                                block_bytes, &empty);
    if (st != Q4_OK)
        return st;
    if (splits < 0)
        return Q4_ERR_SHAPE;
    if (empty)
        return Q4_OK;
    st = q4v::check_workspace(q4v::gemv_splitk_workspace_bytes(M, N, K, splits, block_bytes), a,
                              sizeof(float), w_q, w_bytes, y, M, N, K, workspace, workspace_bytes);
    if (st != Q4_OK)
        return st;
    return launched(q4k::launch_gemv_splitk(fmt, a, static_cast<const uint8_t *>(w_q), y, M, N, K,
                                            q4v::gemv_split_plan(M, N, K, splits, block_bytes),
                                            workspace, as_stream(stream)));
}

static int gemv_prepare(q4k::WeightFormat fmt, const float *a, int M, int K, void *prep,
                        size_t prep_bytes, void *stream)
{
    bool empty = false;
    int st = q4v::check_gemv_prepare(a, M, K, prep, prep_bytes, &empty);
    if (st != Q4_OK || empty)
        return st;
    return launched(q4k::launch_gemv_prepare(fmt, a, prep, M, K, as_stream(stream)));
}

static int gemv_prepared(q4k::WeightFormat fmt, size_t block_bytes, const void *prep,
                         size_t prep_bytes, const void *w_q, size_t w_bytes, float *y, int M,
                         int N, int K, void *stream)
{
    bool empty = false;
    int st = q4v::check_gemv_prepared(prep, prep_bytes, w_q, w_bytes, y, M, N, K, block_bytes,
                                      &empty);
    if (st != Q4_OK || empty)
        return st;
    return launched(q4k::launch_gemv_prepared(fmt, prep, static_cast<const uint8_t *>(w_q), y, M,
                                              N, K, as_stream(stream)));
}

static int gemv_bf16(q4k::WeightFormat fmt, size_t block_bytes, const uint16_t *a,
                     const void *w_q, size_t w_bytes, float *y, int M, int N, int K, void *stream)
{
    bool empty = false;
    int st = q4v::check_product(a, 2, w_q, w_bytes, y, M, N, K, Q4_GEMV_MAX_ROWS, block_bytes,
                                &empty);
    if (st != Q4_OK || empty)
        return st;
    return launched(q4k::launch_gemv_bf16(fmt, a, static_cast<const uint8_t *>(w_q), y, M, N, K,
                                          as_stream(stream)));
}

static int gemv_q8a(q4k::WeightFormat fmt, size_t block_bytes, const void *a_q, size_t a_bytes,
                    const void *w_q, size_t w_bytes, float *y, int M, int N, int K, void *stream)
{
    bool empty = false;
    int st = q4v::check_product_q8a(a_q, a_bytes, w_q, w_bytes, y, M, N, K, Q4_GEMV_MAX_ROWS,
                                    block_bytes, &empty);
    if (st != Q4_OK || empty)
        return st;
    return launched(q4k::launch_gemv_q8a(fmt, static_cast<const uint8_t *>(a_q),
                                         static_cast<const uint8_t *>(w_q), y, M, N, K,
                                         as_stream(stream)));
}

static int gemm_q8a(q4k::WeightFormat fmt, size_t block_bytes, const void *a_q, size_t a_bytes,
                    const void *w_q, size_t w_bytes, float *y, int M, int N, int K,
                    void *workspace, size_t workspace_bytes, void *stream)
{
    bool empty = false;
    int st = q4v::check_product_q8a(a_q, a_bytes, w_q, w_bytes, y, M, N, K, 0, block_bytes,
                                    &empty);
    if (st != Q4_OK || empty)
        return st;
    st = q4v::check_workspace_span(q4v::gemm_q8a_workspace_bytes(M, N, K), a_q, a_bytes, w_q,
                                   w_bytes, y, M, N, workspace, workspace_bytes);
    if (st != Q4_OK)
        return st;
    return launched(q4k::launch_gemm_q8a(fmt, static_cast<const uint8_t *>(a_q),
                                         static_cast<const uint8_t *>(w_q), y, M, N, K, workspace,
                                         as_stream(stream)));
}

static int gemm_bf16(q4k::WeightFormat fmt, size_t block_bytes, const uint16_t *a,
                     const void *w_q, size_t w_bytes, float *y, int M, int N, int K,
                     void *workspace, size_t workspace_bytes, void *stream)
{
    bool empty = false;
    int st = q4v::check_product(a, 2, w_q, w_bytes, y, M, N, K, 0, block_bytes, &empty);
    if (st != Q4_OK || empty)
        return st;
    st = q4v::check_workspace(q4v::gemm_bf16_workspace_bytes(M, N, K), a, 2, w_q, w_bytes, y, M,
                              N, K, workspace, workspace_bytes);
    if (st != Q4_OK)
        return st;
    return launched(q4k::launch_gemm_bf16(fmt, a, static_cast<const uint8_t *>(w_q), y, M, N, K,
                                          workspace, as_stream(stream)));
}

Q4_EXPORT int q4_dequant(const void *w_q, size_t w_bytes, float *out, size_t out_elems, void *stream)
{
    return dequant(q4k::WeightFormat::kQ4_0, 18, w_q, w_bytes, out, out_elems, stream);
}

Q4_EXPORT int q8_dequant(const void *w_q, size_t w_bytes, float *out, size_t out_elems, void *stream)
{
    return dequant(q4k::WeightFormat::kQ8_0, 34, w_q, w_bytes, out, out_elems, stream);
}

Q4_EXPORT int q4_gemv(const float *a, const void *w_q, size_t w_bytes, float *y, int M, int N, int K,
                      void *stream)
{
    return gemv(q4k::WeightFormat::kQ4_0, 18, a, w_q, w_bytes, y, M, N, K, stream);
}

Q4_EXPORT int q8_gemv(const float *a, const void *w_q, size_t w_bytes, float *y, int M, int N, int K,
                      void *stream)
{
    return gemv(q4k::WeightFormat::kQ8_0, 34, a, w_q, w_bytes, y, M, N, K, stream);
}

Q4_EXPORT size_t q4_gemm_workspace_bytes(int M, int N, int K)
{
    return q4v::gemm_workspace_bytes(M, N, K);
}

Q4_EXPORT size_t q8_gemm_workspace_bytes(int M, int N, int K)
{
    return q4v::gemm_workspace_bytes(M, N, K);
}

Q4_EXPORT int q4_gemm(const float *a, const void *w_q, size_t w_bytes, float *y, int M, int N, int K,
                      void *stream)
{
    return gemm_noalloc(q4k::WeightFormat::kQ4_0, 18, a, w_q, w_bytes, y, M, N, K, stream);
}

Q4_EXPORT int q8_gemm(const float *a, const void *w_q, size_t w_bytes, float *y, int M, int N, int K,
                      void *stream)
{
    return gemm_noalloc(q4k::WeightFormat::kQ8_0, 34, a, w_q, w_bytes, y, M, N, K, stream);
}

Q4_EXPORT int q4_gemm_ws(const float *a, const void *w_q, size_t w_bytes, float *y, int M, int N,
                         int K, void *workspace, size_t workspace_bytes, void *stream)
{
    return gemm(q4k::WeightFormat::kQ4_0, 18, a, w_q, w_bytes, y, M, N, K, workspace,
                workspace_bytes, stream);
}

Q4_EXPORT int q8_gemm_ws(const float *a, const void *w_q, size_t w_bytes, float *y, int M, int N,
                         int K, void *workspace, size_t workspace_bytes, void *stream)
{
    return gemm(q4k::WeightFormat::kQ8_0, 34, a, w_q, w_bytes, y, M, N, K, workspace,
                workspace_bytes, stream);
}

Q4_EXPORT int q4_gemv_bf16(const uint16_t *a, const void *w_q, size_t w_bytes, float *y, int M,
                           int N, int K, void *stream)
{
    return gemv_bf16(q4k::WeightFormat::kQ4_0, 18, a, w_q, w_bytes, y, M, N, K, stream);
}

Q4_EXPORT int q8_gemv_bf16(const uint16_t *a, const void *w_q, size_t w_bytes, float *y, int M,
                           int N, int K, void *stream)
{
    return gemv_bf16(q4k::WeightFormat::kQ8_0, 34, a, w_q, w_bytes, y, M, N, K, stream);
}

Q4_EXPORT size_t q4_gemv_prepare_bytes(int M, int K) { return q4v::gemv_prepare_bytes(M, K); }

Q4_EXPORT size_t q8_gemv_prepare_bytes(int M, int K) { return q4v::gemv_prepare_bytes(M, K); }

Q4_EXPORT int q4_gemv_prepare(const float *a, int M, int K, void *prep, size_t prep_bytes,
                              void *stream)
{
    return gemv_prepare(q4k::WeightFormat::kQ4_0, a, M, K, prep, prep_bytes, stream);
}

Q4_EXPORT int q8_gemv_prepare(const float *a, int M, int K, void *prep, size_t prep_bytes,
                              void *stream)
{
    return gemv_prepare(q4k::WeightFormat::kQ8_0, a, M, K, prep, prep_bytes, stream);
}

Q4_EXPORT int q4_gemv_prepared(const void *prep, size_t prep_bytes, const void *w_q,
                               size_t w_bytes, float *y, int M, int N, int K, void *stream)
{
    return gemv_prepared(q4k::WeightFormat::kQ4_0, 18, prep, prep_bytes, w_q, w_bytes, y, M, N, K,
                         stream);
}

Q4_EXPORT int q8_gemv_prepared(const void *prep, size_t prep_bytes, const void *w_q,
                               size_t w_bytes, float *y, int M, int N, int K, void *stream)
{
    return gemv_prepared(q4k::WeightFormat::kQ8_0, 34, prep, prep_bytes, w_q, w_bytes, y, M, N, K,
                         stream);
}

Q4_EXPORT size_t q4_gemv_splitk_workspace_bytes(int M, int N, int K, int splits)
{
    return q4v::gemv_splitk_workspace_bytes(M, N, K, splits, 18);
}

Q4_EXPORT size_t q8_gemv_splitk_workspace_bytes(int M, int N, int K, int splits)
{
    return q4v::gemv_splitk_workspace_bytes(M, N, K, splits, 34);
}

Q4_EXPORT int q4_gemv_splitk(const float *a, const void *w_q, size_t w_bytes, float *y, int M,
                             int N, int K, int splits, void *workspace, size_t workspace_bytes,
                             void *stream)
{
    return gemv_splitk(q4k::WeightFormat::kQ4_0, 18, a, w_q, w_bytes, y, M, N, K, splits,
                       workspace, workspace_bytes, stream);
}

Q4_EXPORT int q8_gemv_splitk(const float *a, const void *w_q, size_t w_bytes, float *y, int M,
                             int N, int K, int splits, void *workspace, size_t workspace_bytes,
                             void *stream)
{
    return gemv_splitk(q4k::WeightFormat::kQ8_0, 34, a, w_q, w_bytes, y, M, N, K, splits,
                       workspace, workspace_bytes, stream);
}

Q4_EXPORT size_t q4_gemm_bf16_workspace_bytes(int M, int N, int K)
{
    return q4v::gemm_bf16_workspace_bytes(M, N, K);
}

Q4_EXPORT size_t q8_gemm_bf16_workspace_bytes(int M, int N, int K)
{
    return q4v::gemm_bf16_workspace_bytes(M, N, K);
}

Q4_EXPORT int q4_gemm_bf16(const uint16_t *a, const void *w_q, size_t w_bytes, float *y, int M,
                           int N, int K, void *workspace, size_t workspace_bytes, void *stream)
{
    return gemm_bf16(q4k::WeightFormat::kQ4_0, 18, a, w_q, w_bytes, y, M, N, K, workspace,
                     workspace_bytes, stream);
}

Q4_EXPORT int q8_gemm_bf16(const uint16_t *a, const void *w_q, size_t w_bytes, float *y, int M,
                           int N, int K, void *workspace, size_t workspace_bytes, void *stream)
{
    return gemm_bf16(q4k::WeightFormat::kQ8_0, 34, a, w_q, w_bytes, y, M, N, K, workspace,
                     workspace_bytes, stream);
}

Q4_EXPORT int q8_quantize(const float *x, size_t n_elems, void *out_q, size_t out_bytes, void *stream)
{
    bool empty = false;
    int st = q4v::check_quantize(x, n_elems, out_q, out_bytes, 34, &empty);
    if (st != Q4_OK || empty)
        return st;
    return launched(q4k::launch_q8_quantize(x, n_elems / 32, static_cast<uint8_t *>(out_q),
                                            as_stream(stream)));
}

Q4_EXPORT int q4_quantize(const float *x, size_t n_elems, void *out_q, size_t out_bytes, void *stream)
{
    bool empty = false;
    int st = q4v::check_quantize(x, n_elems, out_q, out_bytes, 18, &empty);
    if (st != Q4_OK || empty)
        return st;
    return launched(q4k::launch_q4_quantize(x, n_elems / 32, static_cast<uint8_t *>(out_q),
                                            as_stream(stream)));
}

Q4_EXPORT int q4_gemv_q8a(const void *a_q, size_t a_bytes, const void *w_q, size_t w_bytes,
                          float *y, int M, int N, int K, void *stream)
{
    return gemv_q8a(q4k::WeightFormat::kQ4_0, 18, a_q, a_bytes, w_q, w_bytes, y, M, N, K, stream);
}

Q4_EXPORT int q8_gemv_q8a(const void *a_q, size_t a_bytes, const void *w_q, size_t w_bytes,
                          float *y, int M, int N, int K, void *stream)
{
    return gemv_q8a(q4k::WeightFormat::kQ8_0, 34, a_q, a_bytes, w_q, w_bytes, y, M, N, K, stream);
}

Q4_EXPORT size_t q4_gemm_q8a_workspace_bytes(int M, int N, int K)
{
    return q4v::gemm_q8a_workspace_bytes(M, N, K);
}

Q4_EXPORT size_t q8_gemm_q8a_workspace_bytes(int M, int N, int K)
{
    return q4v::gemm_q8a_workspace_bytes(M, N, K);
}

Q4_EXPORT int q4_gemm_q8a(const void *a_q, size_t a_bytes, const void *w_q, size_t w_bytes,
                          float *y, int M, int N, int K, void *workspace, size_t workspace_bytes,
                          void *stream)
{
    return gemm_q8a(q4k::WeightFormat::kQ4_0, 18, a_q, a_bytes, w_q, w_bytes, y, M, N, K,
                    workspace, workspace_bytes, stream);
}

Q4_EXPORT int q8_gemm_q8a(const void *a_q, size_t a_bytes, const void *w_q, size_t w_bytes,
                          float *y, int M, int N, int K, void *workspace, size_t workspace_bytes,
                          void *stream)
{
    return gemm_q8a(q4k::WeightFormat::kQ8_0, 34, a_q, a_bytes, w_q, w_bytes, y, M, N, K,
                    workspace, workspace_bytes, stream);
}

Q4_EXPORT int f8_quantize(const float *x, int M, int K, int block_rows, void *q, size_t q_bytes,
                          float *s, size_t s_elems, void *stream)
{
    bool empty = false;
    int st = q4v::check_f8_codec(x, 4, M, K, block_rows, q, q_bytes, s, s_elems, false, &empty);
    if (st != Q4_OK || empty)
        return st;
    return launched(q4k::launch_f8_quantize(x, static_cast<uint8_t *>(q), s, M, K, block_rows,
                                            as_stream(stream)));
}

Q4_EXPORT int f8_quantize_bf16(const uint16_t *x, int M, int K, int block_rows, void *q,
                               size_t q_bytes, float *s, size_t s_elems, void *stream)
{
    bool empty = false;
    int st = q4v::check_f8_codec(x, 2, M, K, block_rows, q, q_bytes, s, s_elems, false, &empty);
    if (st != Q4_OK || empty)
        return st;
    return launched(q4k::launch_f8_quantize_bf16(x, static_cast<uint8_t *>(q), s, M, K, block_rows,
                                                 as_stream(stream)));
}

Q4_EXPORT int f8_dequant(const void *q, size_t q_bytes, const float *s, size_t s_elems, int M,
                         int K, int block_rows, float *out, size_t out_elems, void *stream)
{
    bool empty = false;
    int st = q4v::check_f8_codec(out, 4, M, K, block_rows, q, q_bytes, s, s_elems, true, &empty);
    if (st != Q4_ERR_SHAPE && out_elems != q_bytes)   // q_bytes is M K, or the size error is its own
        return Q4_ERR_SIZE;
    if (st != Q4_OK || empty)
        return st;
    return launched(q4k::launch_f8_dequant(static_cast<const uint8_t *>(q), s, out, M, K,
                                           block_rows, as_stream(stream)));
}

static int f8_product(const uint8_t *a, const float *a_s, const uint8_t *w, size_t w_bytes,
                      const float *w_s, uint16_t *y, int M, int N, int K, int max_rows, void *stream)
{
    bool empty = false;
    int st = q4v::check_f8_product(a, a_s, w, w_bytes, w_s, y, M, N, K, max_rows, &empty);
    if (st != Q4_OK || empty)
        return st;
    return launched(q4k::launch_f8_gemm(a, a_s, w, w_s, y, M, N, K, as_stream(stream)));
}

Q4_EXPORT int f8_gemm(const uint8_t *a, const float *a_s, const uint8_t *w, size_t w_bytes,
                      const float *w_s, uint16_t *y, int M, int N, int K, void *stream)
{
    return f8_product(a, a_s, w, w_bytes, w_s, y, M, N, K, 0, stream);
}

Q4_EXPORT int f8_gemv(const uint8_t *a, const float *a_s, const uint8_t *w, size_t w_bytes,
                      const float *w_s, uint16_t *y, int M, int N, int K, void *stream)
{
    return f8_product(a, a_s, w, w_bytes, w_s, y, M, N, K, Q4_GEMV_MAX_ROWS, stream);
}

Q4_EXPORT size_t q4_route_workspace_bytes(int T, int E, int top_k)
{
    return q4v::route_workspace_bytes(T, E, top_k);
}

Q4_EXPORT int q4_route(const float *logits, int T, int E, int top_k, int renorm, int32_t *ids,
                       float *weights, int32_t *offsets, int32_t *order, void *workspace,
                       size_t workspace_bytes, void *stream)
{
    bool empty = false;
    int st = q4v::check_route(logits, nullptr, T, E, top_k, ids, weights, offsets, order, workspace,
                              workspace_bytes, q4v::route_workspace_bytes(T, E, top_k), &empty);
    if (st != Q4_OK || empty)
        return st;
    return launched(q4k::launch_route(logits, ids, weights, offsets, order, workspace, T, E, top_k,
                                      renorm != 0, as_stream(stream)));
}

Q4_EXPORT int q4_route_groups(const float *logits, const float *bias, int T, int E, int top_k, int score,
                              int n_groups, int top_groups, int group_best, int renorm, float scale,
                              int32_t *ids, float *weights, int32_t *offsets, int32_t *order,
                              void *workspace, size_t workspace_bytes, void *stream)
{
    int st = q4v::check_route_groups(E, top_k, score, n_groups, top_groups, group_best, scale);
    if (st != Q4_OK)
        return st;
    bool empty = false;
    st = q4v::check_route(logits, bias, T, E, top_k, ids, weights, offsets, order, workspace,
                          workspace_bytes, q4v::route_workspace_bytes(T, E, top_k), &empty);
    if (st != Q4_OK || empty)
        return st;
    const q4k::RouteGroups g = {bias, score == Q4_SCORE_SIGMOID, renorm != 0, n_groups, top_groups,
                                group_best, scale};
    return launched(q4k::launch_route_groups(logits, g, ids, weights, offsets, order, workspace, T, E,
                                             top_k, as_stream(stream)));
}

static int gemm_grouped(q4k::WeightFormat fmt, size_t block_bytes, bool bf16, const void *a,
                        const void *w_q, size_t w_bytes, const int32_t *offsets,
                        const int32_t *order, int share, float *y, int G, int M, int N, int K,
                        void *workspace, size_t workspace_bytes, void *stream)
{
    int st = q4v::check_group_shape(G, M, N, K, 64, 1 << 22, share);
    if (st != Q4_OK)
        return st;
    // G <= 2^10, N < 2^31, K <= 2^22: the counts fit 64 bits.
    if (w_bytes != (size_t)G * (size_t)N * ((size_t)(K / 32) * block_bytes))
        return Q4_ERR_SIZE;
    if (M == 0 || N == 0)
        return Q4_OK;
    const size_t a_rows = ((size_t)M - 1) / (size_t)share + 1;
    const q4v::GroupedArgs g = {a, a_rows * (size_t)K * (bf16 ? 2 : 4), nullptr, 0, w_q, w_bytes,
                                nullptr, 0, offsets, order, y, (size_t)M * (size_t)N * 4, G, M};
    st = q4v::check_grouped(g);
    if (st == Q4_OK)
        st = q4v::check_grouped_workspace(g, q4v::grouped_workspace_bytes(G, M, N, K, block_bytes, bf16 ? 2 : 4),
                                          workspace, workspace_bytes);
    if (st != Q4_OK)
        return st;
    return launched(q4k::launch_gemm_grouped(fmt, bf16, a, static_cast<const uint8_t *>(w_q), offsets,
                                             order, share, y, G, M, N, K, workspace,
                                             as_stream(stream)));
}

Q4_EXPORT int q4_gemm_grouped(const float *a, const void *w_q, size_t w_bytes, const int32_t *offsets,
                              const int32_t *order, int share, float *y, int G, int M, int N, int K,
                              void *workspace, size_t workspace_bytes, void *stream)
{
    return gemm_grouped(q4k::WeightFormat::kQ4_0, 18, false, a, w_q, w_bytes, offsets, order, share, y, G,
                        M, N, K, workspace, workspace_bytes, stream);
}

Q4_EXPORT size_t q4_gemm_grouped_workspace_bytes(int G, int M, int N, int K)
{
    return q4v::grouped_workspace_bytes(G, M, N, K, 18, 4);
}

Q4_EXPORT int q4_gemm_grouped_bf16(const uint16_t *a, const void *w_q, size_t w_bytes, const int32_t *offsets,
                                   const int32_t *order, int share, float *y, int G, int M, int N, int K,
                                   void *workspace, size_t workspace_bytes, void *stream)
{
    return gemm_grouped(q4k::WeightFormat::kQ4_0, 18, true, a, w_q, w_bytes, offsets, order, share, y, G,
                        M, N, K, workspace, workspace_bytes, stream);
}

Q4_EXPORT size_t q4_gemm_grouped_bf16_workspace_bytes(int G, int M, int N, int K)
{
    return q4v::grouped_workspace_bytes(G, M, N, K, 18, 2);
}

Q4_EXPORT int q8_gemm_grouped(const float *a, const void *w_q, size_t w_bytes, const int32_t *offsets,
                              const int32_t *order, int share, float *y, int G, int M, int N, int K,
                              void *workspace, size_t workspace_bytes, void *stream)
{
    return gemm_grouped(q4k::WeightFormat::kQ8_0, 34, false, a, w_q, w_bytes, offsets, order, share, y, G,
                        M, N, K, workspace, workspace_bytes, stream);
}

Q4_EXPORT size_t q8_gemm_grouped_workspace_bytes(int G, int M, int N, int K)
{
    return q4v::grouped_workspace_bytes(G, M, N, K, 34, 4);
}

Q4_EXPORT int q8_gemm_grouped_bf16(const uint16_t *a, const void *w_q, size_t w_bytes, const int32_t *offsets,
                                   const int32_t *order, int share, float *y, int G, int M, int N, int K,
                                   void *workspace, size_t workspace_bytes, void *stream)
{
    return gemm_grouped(q4k::WeightFormat::kQ8_0, 34, true, a, w_q, w_bytes, offsets, order, share, y, G,
                        M, N, K, workspace, workspace_bytes, stream);
}

Q4_EXPORT size_t q8_gemm_grouped_bf16_workspace_bytes(int G, int M, int N, int K)
{
    return q4v::grouped_workspace_bytes(G, M, N, K, 34, 2);
}

Q4_EXPORT int f8_gemm_grouped(const uint8_t *a, const float *a_s, const uint8_t *w, size_t w_bytes,
                              const float *w_s, const int32_t *offsets, const int32_t *order,
                              int share, uint16_t *y, int G, int M, int N, int K, void *stream)
{
    int st = q4v::check_group_shape(G, M, N, K, 32, F8_MAX_K, share);
    const size_t a_rows = st == Q4_OK && M > 0 ? ((size_t)M - 1) / (size_t)share + 1 : 0;
    if (st == Q4_OK && a_rows * (size_t)K >= ((size_t)1 << 31))
        st = Q4_ERR_SHAPE;
    if (st != Q4_OK)
        return st;
    if (w_bytes != (size_t)G * (size_t)N * (size_t)K)
        return Q4_ERR_SIZE;
    if (M == 0 || N == 0)
        return Q4_OK;
    const size_t kb = q4v::f8_blocks(K);
    const q4v::GroupedArgs g = {a, a_rows * (size_t)K, a_s, a_rows * kb * 4, w, w_bytes, w_s,
                                (size_t)G * q4v::f8_blocks(N) * kb * 4, offsets, order, y,
                                (size_t)M * (size_t)N * 2, G, M};
    st = q4v::check_grouped(g);
    if (st != Q4_OK)
        return st;
    return launched(q4k::launch_f8_gemm_grouped(a, a_s, w, w_s, offsets, order, share, y, G, M, N, K,
                                                as_stream(stream)));
}

// The norms: `out` says the form's pointers and sizes.
static int norm(bool bf16, q4k::RowForm form, const q4v::RowsOut &out, const void *x, const float *weights,
                int share, const void *residual, void *sum, const float *gamma, float eps, void *dense,
                void *y, float *s, int M, int K, void *stream)
{
    const q4v::NormCheck c = {x, weights, share, residual, sum, gamma, eps, dense, out, M, K, bf16 ? 2u : 4u};
    bool empty = false;
    int st = q4v::check_norm(c, &empty);
    if (st != Q4_OK || empty)
        return st;
    const q4k::NormArgs a = {x, weights, share, residual, sum, gamma, eps, dense, {y, s}, M, K};
    return launched(q4k::launch_norm(bf16, form, a, as_stream(stream)));
}

static int norm_values(bool bf16, const void *x, const float *weights, int share, const void *residual,
                       void *sum, const float *gamma, float eps, void *y, int y_bf16, int M, int K, void *stream)
{
    return norm(bf16, y_bf16 ? q4k::RowForm::kBf16 : q4k::RowForm::kF32, {y, y_bf16 ? 2u : 4u, false, 0, nullptr, 0},
                x, weights, share, residual, sum, gamma, eps, nullptr, y, nullptr, M, K, stream);
}

Q4_EXPORT int q4_norm(const float *x, const float *weights, int share, const float *residual, float *sum,
                      const float *gamma, float eps, void *y, int y_bf16, int M, int K, void *stream)
{
    return norm_values(false, x, weights, share, residual, sum, gamma, eps, y, y_bf16, M, K, stream);
}

Q4_EXPORT int q4_norm_bf16(const uint16_t *x, const float *weights, int share, const uint16_t *residual,
                           uint16_t *sum, const float *gamma, float eps, void *y, int y_bf16, int M, int K,
                           void *stream)
{
    return norm_values(true, x, weights, share, residual, sum, gamma, eps, y, y_bf16, M, K, stream);
}

Q4_EXPORT int q8_norm(const float *x, const float *weights, int share, const float *residual, float *sum,
                      const float *gamma, float eps, float *y, void *out_q, size_t out_bytes, int M, int K,
                      void *stream)
{
    return norm(false, q4k::RowForm::kQ8_0, {out_q, 0, false, out_bytes, nullptr, 0}, x, weights, share, residual,
                sum, gamma, eps, y, out_q, nullptr, M, K, stream);
}

Q4_EXPORT int q8_norm_bf16(const uint16_t *x, const float *weights, int share, const uint16_t *residual,
                           uint16_t *sum, const float *gamma, float eps, uint16_t *y, void *out_q,
                           size_t out_bytes, int M, int K, void *stream)
{
    return norm(true, q4k::RowForm::kQ8_0, {out_q, 0, false, out_bytes, nullptr, 0}, x, weights, share, residual,
                sum, gamma, eps, y, out_q, nullptr, M, K, stream);
}

Q4_EXPORT int f8_norm(const float *x, const float *weights, int share, const float *residual, float *sum,
                      const float *gamma, float eps, float *y, void *q, size_t q_bytes, float *s,
                      size_t s_elems, int M, int K, void *stream)
{
    return norm(false, q4k::RowForm::kE4M3, {q, 0, true, q_bytes, s, s_elems}, x, weights, share, residual, sum,
                gamma, eps, y, q, s, M, K, stream);
}

Q4_EXPORT int f8_norm_bf16(const uint16_t *x, const float *weights, int share, const uint16_t *residual,
                           uint16_t *sum, const float *gamma, float eps, uint16_t *y, void *q, size_t q_bytes,
                           float *s, size_t s_elems, int M, int K, void *stream)
{
    return norm(true, q4k::RowForm::kE4M3, {q, 0, true, q_bytes, s, s_elems}, x, weights, share, residual, sum,
                gamma, eps, y, q, s, M, K, stream);
}

static int act_rows(bool bf16, q4k::RowForm form, const q4v::RowsOut &out, const void *gate, const void *up, int ld,
                    int act, void *y, float *s, int M, int K, void *stream)
{
    const q4v::ActCheck c = {gate, up, ld, act, out, M, K, bf16 ? 2u : 4u};
    bool empty = false;
    int st = q4v::check_act(c, &empty);
    if (st != Q4_OK || empty)
        return st;
    const q4k::ActArgs a = {gate, up, ld, act, {y, s}, M, K};
    return launched(q4k::launch_act(bf16, form, a, as_stream(stream)));
}

static int act_values(bool bf16, const void *gate, const void *up, int ld, int act, void *y, int y_bf16, int M,
                      int K, void *stream)
{
    return act_rows(bf16, y_bf16 ? q4k::RowForm::kBf16 : q4k::RowForm::kF32,
                    {y, y_bf16 ? 2u : 4u, false, 0, nullptr, 0}, gate, up, ld, act, y, nullptr, M, K, stream);
}

Q4_EXPORT int q4_act(const float *gate, const float *up, int ld, int act, void *y, int y_bf16, int M, int K,
                     void *stream)
{
    return act_values(false, gate, up, ld, act, y, y_bf16, M, K, stream);
}

Q4_EXPORT int q4_act_bf16(const uint16_t *gate, const uint16_t *up, int ld, int act, void *y, int y_bf16, int M,
                          int K, void *stream)
{
    return act_values(true, gate, up, ld, act, y, y_bf16, M, K, stream);
}

Q4_EXPORT int q8_act(const float *gate, const float *up, int ld, int act, void *out_q, size_t out_bytes, int M,
                     int K, void *stream)
{
    return act_rows(false, q4k::RowForm::kQ8_0, {out_q, 0, false, out_bytes, nullptr, 0}, gate, up, ld, act, out_q,
                    nullptr, M, K, stream);
}

Q4_EXPORT int q8_act_bf16(const uint16_t *gate, const uint16_t *up, int ld, int act, void *out_q,
                          size_t out_bytes, int M, int K, void *stream)
{
    return act_rows(true, q4k::RowForm::kQ8_0, {out_q, 0, false, out_bytes, nullptr, 0}, gate, up, ld, act, out_q,
                    nullptr, M, K, stream);
}

Q4_EXPORT int f8_act(const float *gate, const float *up, int ld, int act, void *q, size_t q_bytes, float *s,
                     size_t s_elems, int M, int K, void *stream)
{
    return act_rows(false, q4k::RowForm::kE4M3, {q, 0, true, q_bytes, s, s_elems}, gate, up, ld, act, q, s, M, K,
                    stream);
}

Q4_EXPORT int f8_act_bf16(const uint16_t *gate, const uint16_t *up, int ld, int act, void *q, size_t q_bytes,
                          float *s, size_t s_elems, int M, int K, void *stream)
{
    return act_rows(true, q4k::RowForm::kE4M3, {q, 0, true, q_bytes, s, s_elems}, gate, up, ld, act, q, s, M, K,
                    stream);
}
