// The residual's addition and the root-mean-square norm before a product:
//   h = residual + sum_j w_j x_j,  y = h / sqrt(mean(h^2) + eps) * gamma,
// with y in the form the product reads (rows_out.h) and h as the next residual.
//
// Bound by bytes when there are many rows and by latency when there are few, so
// a row is read once: RW wavefronts hold it in registers, V 16-byte pieces a
// lane, between the sum of its squares and its results. Wavefront w's lane l
// takes pieces (i RW + w) 64 + l, so that a wavefront reads whole lines.
//
// The experts' rows are added in f64 (products of two f32 are exact there, so h
// is the exact sum rounded once but for sums that cancel past 2^-53), and so are
// the squares: two full-rate f64 operations an element, a fortieth of the time
// its bytes take, and the result does not depend on the order of the sums but in
// one row of some 10^7. f32 sums instead are 1 to 4 % faster on every size measured.
//
// Measured, with cold rows: 2048 x 4096, two experts' f32 rows and a residual to
// bfloat16, 25.9 us, 5.9 TB/s (a plain stream of the same bytes 25.9); 1001 x 4096
// bfloat16 to E4M3 7.6 us (5.4); one row 3.0 us (2.2).
#include "f64.h"
#include "launch.h"
#include "rows_out.h"

#include <type_traits>

namespace q4k {

// SUB rows share a wavefront (then RW and V are 1): rows of up to 64 / SUB pieces,
// such as the heads of an attention layer in an array of their own (65536 x 128
// bfloat16 without a residual: 7.8 us, 4.3 TB/s; a wavefront a row 17.4; with a
// residual and the sum 13.4, 5.0 TB/s).
template <class T, RowForm O, bool COMBINE, int RW, int V, int SUB>
__global__ __launch_bounds__(RW < 4 ? 256 : 64 * RW) void k_norm(NormArgs a, double inv_k, int first)
{
    static_assert(SUB == 1 || (RW == 1 && V == 1), "whole rows in a piece a lane");
    constexpr int P = kPiece<T>, WAVES = RW < 4 ? 4 / RW : 1, ROWS = WAVES * SUB, LANES = 64 / SUB;
    __shared__ double part[WAVES][RW];
    const int lane = threadIdx.x & (LANES - 1), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int w = wave % RW, slot = wave / RW;
    const long long want = ((long long)blockIdx.x + first) * ROWS + (SUB > 1 ? (int)threadIdx.x / LANES : slot);
    const size_t row = (size_t)(want < a.M ? want : a.M - 1);   // the last rows' spare lanes write nothing
    const bool live = want < a.M;

    const T *x = static_cast<const T *>(a.x) + row * (size_t)a.share * (size_t)a.K;
    // Without a residual its loads repeat x's: unconditional loads stay in flight together.
    const T *res = a.residual ? static_cast<const T *>(a.residual) + row * (size_t)a.K : x;
    int col[V];
    bool in[V];
    float h[V][P], gamma[V][P];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = ((i * RW + w) * LANES + lane) * P;
        in[i] = c < a.K;
        col[i] = in[i] ? c : 0;
    }
    // gamma is fetched after the rows, or before them where their sum is a loop and the
    // registers allow it.
    const auto get_gamma = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int q = 0; q < P / 4; ++q) {
                const f32x4 g = *reinterpret_cast<const f32x4 *>(a.gamma + col[i] + 4 * q);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    gamma[i][4 * q + k] = g[k];
            }
    };
    constexpr bool kGammaFirst = COMBINE && V == 1;
    if constexpr (kGammaFirst)
        get_gamma();
    if constexpr (COMBINE) {
        float r[V][P];
#pragma unroll
        for (int i = 0; i < V; ++i)
            load_piece(res + col[i], r[i]);
        const float *weights = a.weights ? a.weights + row * (size_t)a.share : nullptr;
        double acc[V][P] = {};
        // Rows of weight 0 (which may hold NaN) add nothing: by a branch over the row in
        // wide workgroups, whose rows' operations count (64 x 7168 bfloat16 of 8 7.6 us,
        // 8.2 by a select an element; 781 x 10240 f32 of 2 33.7, 35.5), else by selects
        // (37 x 4096 f32 of 2 4.2 us, 4.4 by a branch).
        constexpr bool kSkip = P == 8 ? RW >= 8 : RW >= 10 && V > 1;
        // Rows j to j + N - 1.
        const auto add = [&](auto count, int j) __attribute__((always_inline)) {
            constexpr int N = decltype(count)::value;
            float v[N][V][P], w[N];
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int i = 0; i < V; ++i)
                    load_piece(x + (size_t)(j + n) * (size_t)a.K + col[i], v[n][i]);
#pragma unroll
            for (int n = 0; n < N; ++n)
                w[n] = weights ? weights[j + n] : 1.0f;
#pragma unroll
            for (int n = 0; n < N; ++n) {
                if (kSkip && w[n] == 0.0f)
                    continue;
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int k = 0; k < P; ++k)
                        acc[i][k] = fma((double)w[n], (double)(!kSkip && w[n] == 0.0f ? 0.0f : v[n][i][k]), acc[i][k]);
            }
        };
        // N rows are in flight together, by the row's width alone: as many as leave the
        // registers to two workgroups a compute unit or more, also where there are fewer
        // workgroups than compute units (64 x 7168 bfloat16 of 8, two in flight and 50 of
        // 128 registers used, 7.5 us, some 4 for its bytes). Against one row fetched ahead
        // of the one that is added (us, to E4M3): 976 x 512 bfloat16 of 8 4.8, 7.4; 3906 x
        // 2048 f32 of 2 23.1, 25.1; 558 x 7168 bfloat16 of 4 13.8, 15.2; at worst 279 x
        // 7168 of 8 13.4, 12.3. With eight f32 pieces a lane, or four of bfloat16 (K >
        // 16384), the f64 sums alone fill the registers and some are spilled: 139 x 28672
        // of 4 to E4M3 f32 32.8 us (21 to 39 registers), bfloat16 15.8 (1 to 5).
        constexpr int N = V == 1 ? (P == 4 ? 8 : RW < 10 ? 4 : 2) : V == 2 ? 2 : 1;
        int j = 0;
        for (; j + N <= a.share; j += N)
            add(std::integral_constant<int, N>{}, j);
        if constexpr (N > 4)
            for (; j + 4 <= a.share; j += 4)
                add(std::integral_constant<int, 4>{}, j);
        if constexpr (N > 2)
            for (; j + 2 <= a.share; j += 2)
                add(std::integral_constant<int, 2>{}, j);
        for (; j < a.share; ++j)
            add(std::integral_constant<int, 1>{}, j);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int k = 0; k < P; ++k)
                h[i][k] = (float)(a.residual ? acc[i][k] + (double)r[i][k] : acc[i][k]);
    } else {
        float r[V][P];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            load_piece(x + col[i], h[i]);
            load_piece(res + col[i], r[i]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int k = 0; k < P; ++k)
                h[i][k] = a.residual ? h[i][k] + r[i][k] : h[i][k];
    }
    if constexpr (!kGammaFirst)
        get_gamma();

    // Rows of bfloat16 in one piece a lane write h before they are reduced (1001 x
    // 4096 to E4M3 7.9 us, 8.2 after), the others after (512 x 4096 f32 to Q8_0 6.6
    // us, 7.3 before).
    constexpr bool kEarly = sizeof(T) == 2 && V == 1;
    const auto put_sum = [&]() __attribute__((always_inline)) {
        if (a.sum && live) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (in[i])
                    store_piece(static_cast<T *>(a.sum) + row * (size_t)a.K + col[i], h[i]);
        }
    };
    if constexpr (kEarly)
        put_sum();

    double sq = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        double piece = 0.0;
#pragma unroll
        for (int k = 0; k < P; ++k)
            piece = fma((double)h[i][k], (double)h[i][k], piece);
        sq += in[i] ? piece : 0.0;
    }
    sq = SUB > 1 ? lanes_sum_f64<LANES>(sq) : wave_sum_f64(sq);
    if constexpr (RW > 1) {
        if (lane == 0)
            part[slot][w] = sq;
        __syncthreads();
        sq = part[slot][0];
#pragma unroll
        for (int k = 1; k < RW; ++k)
            sq += part[slot][k];
    }
    const double ms = fma(sq, inv_k, (double)a.eps);
    // Rows below 2^-125, whose 1 / rms leaves f32 (eps is 0 or as small), are scaled
    // up first, and those above 2^125, where it would lose bits below 2^-126, down.
    const bool tiny = ms < 0x1p-250, huge = ms > 0x1p250;
    // 0 of a row of zeros and of one with an infinity, NaN of one with a NaN.
    const float rstd = ms > 0.0 && ms < __builtin_inf() ? (float)(rsqrt_f64(ms) * (tiny ? 0x1p-64 : huge ? 0x1p64 : 1.0))
                       : ms != ms                       ? __builtin_nanf("")
                                                        : 0.0f;
    if constexpr (!kEarly)
        put_sum();

    if (__builtin_expect(tiny || huge, 0)) {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int k = 0; k < P; ++k)
                h[i][k] *= tiny ? 0x1p64f : 0x1p-64f;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int k = 0; k < P; ++k)
            h[i][k] = h[i][k] * rstd * gamma[i][k];
        if (a.dense && live && in[i])
            store_piece(static_cast<T *>(a.dense) + row * (size_t)a.K + col[i], h[i]);
        put_piece<O, LANES>(a.out, a.K, h[i], in[i] && live, row, col[i]);
    }
}

template <class T, RowForm O, bool COMBINE, int RW, int V, int SUB = 1>
static hipError_t launch_rows(const NormArgs &a, hipStream_t st)
{
    constexpr int ROWS = (RW < 4 ? 4 / RW : 1) * SUB;
    return launch_parts(k_norm<T, O, COMBINE, RW, V, SUB>, ((long long)a.M + ROWS - 1) / ROWS, 1, RW < 4 ? 256 : 64 * RW,
                        st, a, 1.0 / a.K);
}

// As many wavefronts a row as take it in one piece a lane: the shortest way for few
// rows, and for many (1001 x 4096 bfloat16 to E4M3 7.6 us with 8 wavefronts a row,
// 8.3 with 4 of two pieces). The widths with 5, 10 and 12 wavefronts beside the
// powers of two leave fewer lanes idle (us, with the next power of two and with
// them): 512 x 2560 bfloat16 to E4M3 4.5 4.2, 512 x 5120 6.7 6.2, 900 x 10240 of 2 to
// Q8_0 27.8 22.4, 512 x 12288 12.2 11.6; at worst 1024 x 5120 f32 of 2 21.4 22.5.
// From 9 to 16 of them the workgroups get so large that two are on a compute unit
// at a time; many rows of those take two pieces a lane in 5 or 8 wavefronts, unless
// experts' rows of bfloat16 are added (1116 x 7168 of 2 to E4M3 16.9, 17.7 us)
// (us, 16 x 1 and 8 x 2; f32):
//                              M = 512     1024        2048
//   4096 to f32                7.2  7.0  14.1 13.1   25.6 23.9
//   4096 to Q8_0               6.7  7.5  12.7 12.0   22.7 21.2
//   4096 to E4M3               7.1  7.3  12.9 11.8   22.6 20.9
//   4096 to bfloat16, of 2                           26.9 25.8
template <class T, RowForm O, bool COMBINE>
static hipError_t launch_width(const NormArgs &a, hipStream_t st)
{
    const int pieces = a.K / kPiece<T>, waves = (pieces + 63) / 64;   // wavefronts of one piece a lane
    if (pieces <= 16)
        return launch_rows<T, O, COMBINE, 1, 1, 4>(a, st);
    if (pieces <= 32)
        return launch_rows<T, O, COMBINE, 1, 1, 2>(a, st);
    if (waves <= 1)
        return launch_rows<T, O, COMBINE, 1, 1>(a, st);
    if (waves <= 2)
        return launch_rows<T, O, COMBINE, 2, 1>(a, st);
    if (waves <= 4)
        return launch_rows<T, O, COMBINE, 4, 1>(a, st);
    if (waves <= 5)
        return launch_rows<T, O, COMBINE, 5, 1>(a, st);
    if (waves <= 8)
        return launch_rows<T, O, COMBINE, 8, 1>(a, st);
    if (waves <= 16) {
        if constexpr (!COMBINE || kPiece<T> == 4)
            if (a.M >= 1024)
                return waves <= 10 ? launch_rows<T, O, COMBINE, 5, 2>(a, st) : launch_rows<T, O, COMBINE, 8, 2>(a, st);
        return waves <= 10   ? launch_rows<T, O, COMBINE, 10, 1>(a, st)
               : waves <= 12 ? launch_rows<T, O, COMBINE, 12, 1>(a, st)
                             : launch_rows<T, O, COMBINE, 16, 1>(a, st);
    }
    if (waves <= 20)
        return launch_rows<T, O, COMBINE, 10, 2>(a, st);
    if (waves <= 24)
        return launch_rows<T, O, COMBINE, 12, 2>(a, st);
    if (waves <= 32)
        return launch_rows<T, O, COMBINE, 16, 2>(a, st);
    if (waves <= 64)
        return launch_rows<T, O, COMBINE, 16, 4>(a, st);
    if constexpr (kPiece<T> == 4)
        return launch_rows<T, O, COMBINE, 16, 8>(a, st);
    return hipErrorInvalidValue;   // K <= Q4_NORM_MAX_K ends above
}

template <class T, RowForm O>
static hipError_t launch_form(const NormArgs &a, hipStream_t st)
{
    return a.share > 1 || a.weights ? launch_width<T, O, true>(a, st) : launch_width<T, O, false>(a, st);
}

template <class T>
static hipError_t launch_type(RowForm form, const NormArgs &a, hipStream_t st)
{
    switch (form) {
    case RowForm::kF32: return launch_form<T, RowForm::kF32>(a, st);
    case RowForm::kBf16: return launch_form<T, RowForm::kBf16>(a, st);
    case RowForm::kQ8_0: return launch_form<T, RowForm::kQ8_0>(a, st);
    default: return launch_form<T, RowForm::kE4M3>(a, st);
    }
}

hipError_t launch_norm(bool bf16, RowForm form, const NormArgs &a, hipStream_t st)
{
    return bf16 ? launch_type<uint16_t>(form, a, st) : launch_type<float>(form, a, st);
}

}  // namespace q4k
