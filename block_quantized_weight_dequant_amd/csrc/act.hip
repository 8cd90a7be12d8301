// The gated activation between two products: y = f(gate) up, f SiLU or GELU (tanh
// form), y in the form the next product reads (rows_out.h).
//
// Bound by bytes. A wavefront takes 64 V pieces of one row (C wavefronts of a
// workgroup side by side, 4 / C rows), so that its loads and stores are whole
// lines and a block's maximum stays within it.
//
// f(g) = g / (1 + exp(-z)), z = g for SiLU and 2 sqrt(2 / pi) (g + 0.044715 g^3)
// for GELU (where (1 + tanh u) / 2 = 1 / (1 + exp(-2 u))): one exponential and one
// reciprocal, both from the hardware's f32 instructions (1 unit in the last
// place). exp(-z) is 2^(hi + lo), hi = -z log2 e rounded and lo its remainder, which
// keeps the rounding of a large exponent out of the result.
#include "launch.h"
#include "rows_out.h"

namespace q4k {

template <int ACT>
__device__ __forceinline__ float gate_value(float g)
{
    float z = g;
    if constexpr (ACT == Q4_ACT_GELU)
        z = g * fmaf(g * g, (float)(1.5957691216057308 * 0.044715), 1.5957691216057308f);
    z = __builtin_amdgcn_fmed3f(z, -130.0f, 130.0f);   // past them e is 0 or infinite either way
    constexpr float kLog2e = 1.44269504f, kLog2eLo = 1.92596303e-8f;   // log2 e = kLog2e + kLog2eLo
    const float hi = -z * kLog2e;
    const float lo = fmaf(-z, kLog2e, -hi) - z * kLog2eLo;
    const float e = __builtin_amdgcn_exp2f(hi);
    // e 2^lo = e + e lo ln 2 to within lo^2 / 2; where e is infinite the product with
    // lo may not be taken (0 times it is NaN).
    const float p = e < 0x1p126f ? fmaf(e, lo * 0.693147181f, e) : e;
    return g * __builtin_amdgcn_rcpf(1.0f + p);
}

template <class T, RowForm O, int ACT, int C, int V>
__global__ __launch_bounds__(256) void k_act(ActArgs a, int first)
{
    constexpr int P = kPiece<T>, ROWS = 4 / C;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const long long row = ((long long)blockIdx.x + first) * ROWS + wave / C;
    if (row >= a.M)
        return;
    const T *gate = static_cast<const T *>(a.gate) + (size_t)row * (size_t)a.ld;
    const T *up = a.up ? static_cast<const T *>(a.up) + (size_t)row * (size_t)a.ld : gate;
    int col[V];
    bool in[V];
    float g[V][P], u[V][P];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const long long c = (((long long)blockIdx.y * C + wave % C) * V + i) * 64 * P + lane * P;
        in[i] = c < a.K;
        col[i] = in[i] ? (int)c : 0;
        load_piece(gate + col[i], g[i]);
        load_piece(up + col[i], u[i]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int k = 0; k < P; ++k) {
            const float f = gate_value<ACT>(g[i][k]);
            g[i][k] = in[i] ? (a.up ? f * u[i][k] : f) : 0.0f;
        }
        put_piece<O>(a.out, a.K, g[i], in[i], (size_t)row, col[i]);
    }
}

template <class T, RowForm O, int ACT>
static hipError_t launch_f(const ActArgs &a, hipStream_t st)
{
    constexpr int V = 1;
    const long long waves = ((long long)a.K / kPiece<T> + 64 * V - 1) / (64 * V);
    const auto go = [&](auto kernel, int c) {
        const long long rows = 4 / c;
        return launch_parts(kernel, (a.M + rows - 1) / rows, (unsigned)((waves + c - 1) / c), 256, st, a);
    };
    return waves <= 1 ? go(k_act<T, O, ACT, 1, V>, 1) : waves <= 2 ? go(k_act<T, O, ACT, 2, V>, 2) : go(k_act<T, O, ACT, 4, V>, 4);
}

template <class T, RowForm O>
static hipError_t launch_form(const ActArgs &a, hipStream_t st)
{
    return a.act == Q4_ACT_GELU ? launch_f<T, O, Q4_ACT_GELU>(a, st) : launch_f<T, O, Q4_ACT_SILU>(a, st);
}

template <class T>
static hipError_t launch_type(RowForm form, const ActArgs &a, hipStream_t st)
{
    switch (form) {
    case RowForm::kF32: return launch_form<T, RowForm::kF32>(a, st);
    case RowForm::kBf16: return launch_form<T, RowForm::kBf16>(a, st);
    case RowForm::kQ8_0: return launch_form<T, RowForm::kQ8_0>(a, st);
    default: return launch_form<T, RowForm::kE4M3>(a, st);
    }
}

hipError_t launch_act(bool bf16, RowForm form, const ActArgs &a, hipStream_t st)
{
    return bf16 ? launch_type<uint16_t>(form, a, st) : launch_type<float>(form, a, st);
}

}  // namespace q4k
