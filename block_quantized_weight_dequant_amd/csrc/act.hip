// The gated activation between two products: y = f(gate) up, f SiLU or GELU (tanh
// form), y in the form the next product reads (rows_out.h).
//
// Bound by bytes, with some 25 operations an element close behind. A lane takes one
// 16-byte piece (two or four take 9 % longer), and the lanes of a block of the
// output go to the blocks of all rows in turn, so that no lane idles at the end of
// a row and a block's maximum stays within its lanes. With whole wavefronts, or
// workgroups, in one row instead, 4096 x 2816 bfloat16 to E4M3 takes 13.4 us, or
// 16.9, for 12.0. 4096 x 14336 bfloat16 to E4M3: 48.9 us, 6.0 TB/s; 1001 x 14336 f32
// to bfloat16 24.1 us, 5.9 TB/s; plain streams of the same bytes take 47.6 and 24.1.
//
// f(g) = g / (1 + exp(-z)), z = g for SiLU and 2 sqrt(2 / pi) (g + 0.044715 g^3)
// for GELU (where (1 + tanh u) / 2 = 1 / (1 + exp(-2 u))): one exponential and one
// reciprocal, both from the hardware's f32 instructions (1 unit in the last
// place, four times the time of another). The reciprocal takes its remainder once
// and is then within a little more than half a unit; it and not the quotient does,
// whose remainder is NaN where g is infinite.
#include "launch.h"
#include "rows_out.h"

namespace q4k {

template <int ACT>
__device__ __forceinline__ float gate_value(float g)
{
    // Below these gates f is nearer to 0 than 2^-119 and counts as f there, so that
    // the exponential stays finite. The maximum keeps NaN.
    g = __builtin_elementwise_maximum(g, ACT == Q4_ACT_GELU ? -9.98f : -87.0f);
    constexpr double kLog2e = 1.4426950408889634, kTwice = 1.5957691216057308;   // 2 sqrt(2 / pi)
    const float hi = ACT == Q4_ACT_GELU ? g * fmaf(g * g, (float)(-kTwice * 0.044715 * kLog2e), (float)(-kTwice * kLog2e))
                                        : g * (float)-kLog2e;   // -z log2 e
    const float d = 1.0f + __builtin_amdgcn_exp2f(hi);
    const float r = __builtin_amdgcn_rcpf(d);
    return g * fmaf(fmaf(-d, r, 1.0f), r, r);
}

// Columns of a block of the output; K is a multiple of 32.
template <RowForm O>
constexpr int kActBlock = O == RowForm::kE4M3 ? 128 : 32;

// Block i of a launch lies in row first + i / blocks; the quotient is i times mul,
// 2^shift / blocks rounded up, shifted: exact for i < 2^31, as mul is too large by
// less than 1 and 2^shift >= 2^31 blocks.
template <class T, RowForm O, int ACT>
__global__ __launch_bounds__(256) void k_act(ActArgs a, uint32_t blocks, uint32_t mul, int shift, int first)
{
    constexpr int P = kPiece<T>, LANES = kActBlock<O> / P;
    const uint32_t i = blockIdx.x * (256u / LANES) + threadIdx.x / LANES, r = (uint32_t)(((uint64_t)i * mul) >> shift);
    const long long row = (long long)first + r;
    if (row >= a.M)
        return;
    const T *gate = static_cast<const T *>(a.gate) + (size_t)row * (size_t)a.ld;
    const T *up = a.up ? static_cast<const T *>(a.up) + (size_t)row * (size_t)a.ld : gate;
    const int c = (int)((i - r * blocks) * LANES + threadIdx.x % LANES) * P;   // K <= 2^22
    const bool in = c < a.K;
    const int col = in ? c : 0;
    float g[P], u[P];
    load_piece(gate + col, g);
    load_piece(up + col, u);
#pragma unroll
    for (int k = 0; k < P; ++k)
        g[k] = gate_value<ACT>(g[k]);
    if (a.up) {
#pragma unroll
        for (int k = 0; k < P; ++k)
            g[k] *= u[k];
    }
    put_piece<O>(a.out, a.K, g, in, (size_t)row, col);
}

template <class T, RowForm O, int ACT>
static hipError_t launch_f(const ActArgs &a, hipStream_t st)
{
    constexpr int LANES = kActBlock<O> / kPiece<T>;
    const int blocks = (a.K + kActBlock<O> - 1) / kActBlock<O>;
    int shift = 31;
    while ((1ll << (shift - 31)) < blocks)
        ++shift;
    const uint32_t mul = (uint32_t)(((1ull << shift) + (uint64_t)blocks - 1) / (uint64_t)blocks);
    // At most 2^28 lanes a launch, 256 rows of the longest.
    const long long part = (1 << 28) / (blocks * LANES);
    hipError_t e = hipSuccess;
    for (long long first = 0; first < a.M && e == hipSuccess; first += part) {
        const long long rows = a.M - first < part ? a.M - first : part;
        e = launch_kernel(k_act<T, O, ACT>, dim3((unsigned)((rows * blocks * LANES + 255) / 256)), dim3(256), 0, st, a,
                          (uint32_t)blocks, mul, shift, (int)first);
    }
    return e;
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
