// What the norm and the activation share: 16-byte pieces of a row of f32 or
// bfloat16, and a row of f32 results written in the form that the next product
// reads (f32, bfloat16, Q8_0 blocks, E4M3 codes with a scale for each 128
// columns).
//
// A lane holds P consecutive elements of a row, 16 bytes of input (P = 4 of f32,
// 8 of bfloat16), and a block's lanes its pieces in order: a Q8_0 block is 32 / P
// neighbouring lanes, a block of 128 columns 128 / P, the first of them at a multiple
// of their number, so that no block leaves its wavefront or straddles the DPP rows
// that its maximum crosses.
#pragma once

#include "device_common.h"
#include "launch.h"

namespace q4k {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr float kE4M3Max = 448.0f;

// Elements of a 16-byte piece.
template <class T>
constexpr int kPiece = 16 / (int)sizeof(T);

// Rows are read once: their loads are non-temporal.
__device__ __forceinline__ void load_piece(const float *p, float (&v)[4])
{
    const f32x4 a = __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(p));
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = a[i];
}
__device__ __forceinline__ void load_piece(const uint16_t *p, float (&v)[8])
{
    const u32x4 a = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(a[i] << 16);
        v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
}

// P values of f32, or rounded to bfloat16, at p (aligned to 16 bytes, to 8
// for four bfloat16 values).
template <class T>
__device__ __forceinline__ void store(void *p, T v)
{
    __builtin_nontemporal_store(v, static_cast<T *>(p));
}
template <int P>
__device__ __forceinline__ void store_piece(float *p, const float (&v)[P])
{
#pragma unroll
    for (int h = 0; h < P / 4; ++h)
        store(p + 4 * h, (f32x4){v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]});
}
template <int P>
__device__ __forceinline__ void store_piece(uint16_t *p, const float (&v)[P])
{
    uint32_t w[P / 2];
#pragma unroll
    for (int h = 0; h < P / 2; ++h)
        w[h] = bitcast<uint32_t>((bf16x2){(__bf16)v[2 * h], (__bf16)v[2 * h + 1]});
    if constexpr (P == 8)
        store(p, (u32x4){w[0], w[1], w[2], w[3]});
    else
        store(p, (u32x2){w[0], w[1]});
}

// x / s for a scale s >= 0 that no |x| exceeds `limit` times by more than a
// rounding, to be rounded to a code. s in [2^-90, 2^90]: from the correctly
// rounded reciprocal and one step with the exact remainder (an FMA), which leaves
// the quotient on the side of every midpoint between two E4M3 values, and of
// every k + 1/2 up to 128, on which the correctly rounded one is, or on it if that
// is: checked for all significands of s, all midpoints (of up to 8 bits) and the nine
// x nearest to each product, beyond which no quotient comes within a unit in the last
// place. No intermediate leaves the normal range here but where the quotient is
// far below the smallest code. The remainder of -0 is +0, which would lose its
// sign: the quotient takes x's. Four operations an element; a division takes
// about twelve. Other scales divide; s == 0 gives 0. clamp: to +-limit there (in
// the range above the quotient is at most a rounding past it, which the codes
// absorb). NaN stays NaN under every scale.
template <int P>
__device__ __forceinline__ void quotients(const float (&x)[P], float s, bool clamp, float limit, float (&q)[P])
{
    if (s >= 0x1p-90f && s <= 0x1p90f) {
        const float r = 1.0f / s;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float q0 = x[i] * r;
            q[i] = __builtin_copysignf(fmaf(fmaf(-q0, s, x[i]), r, q0), x[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float v = x[i] / s;
            q[i] = s == 0.0f ? fabsf(x[i]) * 0.0f
                   : clamp ? __builtin_elementwise_minimum(__builtin_elementwise_maximum(v, -limit), limit) : v;
        }
    }
}

// E4M3 codes of P quotients, four to a dword. The conversion rounds everything
// below 464 to 448 at most.
template <int P>
__device__ __forceinline__ void e4m3_codes(const float (&x)[P], float s, uint32_t (&w)[P / 4])
{
    float q[P];
    quotients(x, s, true, kE4M3Max, q);
#pragma unroll
    for (int h = 0; h < P / 4; ++h) {
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h], q[4 * h + 1], 0, false);
        w[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h + 2], q[4 * h + 3], lo, true);
    }
}

// The larger of two; of NaN and a number the number, or NaN (NAN_WINS).
template <bool NAN_WINS>
__device__ __forceinline__ float larger_of(float a, float b)
{
    if constexpr (NAN_WINS)
        return __builtin_elementwise_maximum(a, b);
    else
        return fmaxf(a, b);
}

template <bool NAN_WINS = false, int P>
__device__ __forceinline__ float abs_max(const float (&v)[P])
{
    float m = fabsf(v[0]);
#pragma unroll
    for (int i = 1; i < P; ++i)
        m = larger_of<NAN_WINS>(m, fabsf(v[i]));
    return m;
}

template <bool NAN_WINS, int CTRL>
__device__ __forceinline__ float dpp_max(float v)
{
    return larger_of<NAN_WINS>(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, false)));
}

// Largest over each L neighbouring lanes (4, 8, 16 or 32), in every one of them.
template <int L, bool NAN_WINS = false>
__device__ __forceinline__ float lanes_max(float v)
{
    v = dpp_max<NAN_WINS, 0xB1>(v);        // quad_perm 1,0,3,2
    v = dpp_max<NAN_WINS, 0x4E>(v);        // quad_perm 2,3,0,1
    if constexpr (L >= 8)
        v = dpp_max<NAN_WINS, 0x141>(v);   // row_half_mirror
    if constexpr (L >= 16)
        v = dpp_max<NAN_WINS, 0x140>(v);   // row_mirror
    if constexpr (L >= 32) {
        // Rows of 16 lanes 0 and 1, and 2 and 3, change places.
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = larger_of<NAN_WINS>(__uint_as_float(r[0]), __uint_as_float(r[1]));
    }
    return v;
}

// max / c, correctly rounded, for c = 448 or 127: the quotient by the reciprocal
// and one step with the exact remainder, checked for every significand (both checks:
// tests/test_quotients.py).
__device__ __forceinline__ float scale_of(float max, float c)
{
    if (!(max >= 0x1p-90f && max <= 0x1p120f))
        return max / c;
    const float r = 1.0f / c, q = max * r;
    return fmaf(fmaf(-q, c, max), r, q);
}

// One piece of row `row` at column col, in the form O. Every lane of a
// block calls it; lanes that are not `in` (past the row's end) count for no
// maximum and write nothing. LANES neighbouring lanes hold a row, where several rows
// share the wavefront (a block is no longer than its row).
template <RowForm O, int LANES = 64, int P>
__device__ __forceinline__ void put_piece(const RowOut &o, int K, const float (&v)[P], bool in, size_t row, int col)
{
    const size_t at = row * (size_t)K + (size_t)col;
    if constexpr (O == RowForm::kF32) {
        if (in)
            store_piece(static_cast<float *>(o.y) + at, v);
    } else if constexpr (O == RowForm::kBf16) {
        if (in)
            store_piece(static_cast<uint16_t *>(o.y) + at, v);
    } else if constexpr (O == RowForm::kE4M3) {
        const float s = scale_of(lanes_max<(128 / P < LANES ? 128 / P : LANES)>(in ? abs_max(v) : 0.0f), kE4M3Max);
        uint32_t w[P / 4];
        e4m3_codes(v, s, w);
        if (in) {
            uint8_t *p = static_cast<uint8_t *>(o.y) + at;
            if constexpr (P == 8)
                store(p, (u32x2){w[0], w[1]});
            else
                store(p, w[0]);
            if ((col & 127) == 0)
                o.s[row * (size_t)(((unsigned)K + 127) / 128) + (size_t)((unsigned)col >> 7)] = s;
        }
    } else {
        // Q8_0: a block's 34 bytes are 2-byte aligned, and so are these stores. Its codes
        // have no NaN, so one in the block is the scale's.
        const float d = scale_of(lanes_max<32 / P, true>(in ? abs_max<true>(v) : 0.0f), 127.0f);
        float q[P];
        quotients(v, d, false, 0.0f, q);
        uint32_t w[P / 4];
#pragma unroll
        for (int h = 0; h < P / 4; ++h) {
            w[h] = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[h] |= (uint32_t)((int)roundf(q[4 * h + i]) & 255) << (8 * i);
        }
        if (in) {
            uint8_t *b = static_cast<uint8_t *>(o.y) + (row * (size_t)((unsigned)K >> 5) + (size_t)((unsigned)col >> 5)) * kQ8Bytes;
            __builtin_memcpy(b + 2 + (col & 31), w, P);
            if ((col & 31) == 0)
                *reinterpret_cast<uint16_t *>(b) = (uint16_t)f32_to_f16_bits(d);
        }
    }
}

}  // namespace q4k
