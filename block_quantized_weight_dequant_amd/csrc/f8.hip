// E4M3 (8-bit floating point, 4 exponent and 3 fraction bits, no infinities,
// largest value 448) with one f32 scale for each block of 128: the quantizers,
// the decode, and the product y = (a_s a) @ (w_s w)^T, also grouped by expert.
//
// Layout: activations are codes [M, K] with scales [M, ceil(K / 128)] (one per
// 128 columns of a row), weights codes [N, K] with scales [ceil(N / 128),
// ceil(K / 128)] (one per 128 x 128 tile), all row-major; a row's last block
// may be short.
#include <algorithm>

#include "device_common.h"
#include "f8_forms.h"
#include "groups.h"
#include "launch.h"
#include "rows_out.h"

namespace q4k {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// Quantize. Per block: s = max|x| / 448 in f32, code = the E4M3 value nearest
// to x / s (ties to even), the quotient rounded once to f32 and clamped to
// +-448; s == 0 stores zeros. s is rounded, so the largest quotient is often a
// step past 448 (448 + 2^-15, one ordinary maximum in twelve), and farther only
// where s is subnormal.
// Bound by the bytes of x: 16 lanes share a block of a row, eight elements
// each, so a wavefront reads four blocks (2 KB of f32) and writes 512 bytes
// of codes in whole lines, and the maximum crosses 16 lanes in four DPP moves.

template <class T>
struct Eight {
    float v[8];
    __device__ __forceinline__ void load(const T *p)
    {
        if constexpr (sizeof(T) == 4) {
            const f32x4 a = *reinterpret_cast<const f32x4 *>(p), b = *reinterpret_cast<const f32x4 *>(p + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = a[i], v[4 + i] = b[i];
        } else {
            const u32x4 a = *reinterpret_cast<const u32x4 *>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(a[i] << 16);
                v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
            }
        }
    }
    __device__ __forceinline__ void clear_if(bool c)
    {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = c ? 0.0f : v[i];
    }
    __device__ __forceinline__ float amax() const
    {
        float m = fabsf(v[0]);
#pragma unroll
        for (int i = 1; i < 8; ++i)
            m = fmaxf(m, fabsf(v[i]));
        return m;
    }
    __device__ __forceinline__ u32x2 codes(float s) const
    {
        uint32_t w[2];
        e4m3_codes(v, s, w);
        return (u32x2){w[0], w[1]};
    }
};

// One scale per 128 columns of a row: 16 blocks per 256-thread workgroup, one a
// thread group (2048 x 4096 bfloat16: 6.4 us, 3.9 TB/s; two or four blocks in
// flight a group, with half and a quarter of the workgroups, take 6.6 and 7.3).
template <class T>
__global__ __launch_bounds__(256) void k_f8_quantize_rows(const T *__restrict__ x,
                                                         uint8_t *__restrict__ q,
                                                         float *__restrict__ s, int K, unsigned Kb,
                                                         unsigned n_blocks)
{
    const unsigned p = threadIdx.x & 15, b = blockIdx.x * 16 + (threadIdx.x >> 4);
    if (b >= n_blocks)   // whole groups of 16 lanes
        return;
    const unsigned row = b / Kb, col = (b - row * Kb) * 128 + 8 * p;
    const bool in = col < (unsigned)K;
    const size_t at = (size_t)row * (size_t)K + (in ? col : 0u);
    Eight<T> v;
    v.load(x + at);
    v.clear_if(!in);
    const float sc = lanes_max<16>(v.amax()) / kE4M3Max;
    if (in)
        *reinterpret_cast<u32x2 *>(q + at) = v.codes(sc);
    if (p == 0)
        s[b] = sc;
}

// One scale per 128 x 128 tile: a workgroup holds the tile in registers
// (eight rows of eight elements a thread) between its maximum and its codes,
// so x is read once.
template <class T>
__global__ __launch_bounds__(256) void k_f8_quantize_tiles(const T *__restrict__ x,
                                                          uint8_t *__restrict__ q,
                                                          float *__restrict__ s, int M, int K,
                                                          int Kb, int first)
{
    __shared__ float wave_max[4];
    const int tid = threadIdx.x;
    const int tile = first + (int)blockIdx.x, rb = tile / Kb, kb = tile - rb * Kb;
    const int col = kb * 128 + 8 * (tid & 15);
    const bool col_in = col < K;
    const T *src = x + (col_in ? col : 0);
    const int row0 = rb * 128 + (tid >> 4);
    Eight<T> v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i].load(src + (size_t)min(row0 + 16 * i, M - 1) * (size_t)K);
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i].clear_if(!col_in || row0 + 16 * i >= M);
        m = fmaxf(m, v[i].amax());
    }
    m = lanes_max<16>(m);
    m = fmaxf(m, __shfl_xor(m, 16));
    m = fmaxf(m, __shfl_xor(m, 32));
    if ((tid & 63) == 0)
        wave_max[tid >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(wave_max[0], wave_max[1]), fmaxf(wave_max[2], wave_max[3]));
    const float sc = m / kE4M3Max;
    if (tid == 0)
        s[tile] = sc;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = row0 + 16 * i;
        if (col_in && row < M)
            *reinterpret_cast<u32x2 *>(q + (size_t)row * (size_t)K + col) = v[i].codes(sc);
    }
}

template <class T>
static hipError_t launch_quantize_t(const T *x, uint8_t *q, float *s, int M, int K, int block_rows,
                                    hipStream_t st)
{
    // At most 2^23 workgroups (2^31 threads) a launch.
    const unsigned Kb = ((unsigned)K + 127) / 128;
    if (block_rows == 1) {
        const int rows = (int)((1u << 27) / Kb);   // K <= 2^31: at least 8
        for (int r0 = 0; r0 < M; r0 += rows) {
            const unsigned nb = (unsigned)(M - r0 < rows ? M - r0 : rows) * Kb;
            const hipError_t e = launch_kernel(k_f8_quantize_rows<T>, dim3((nb + 15) / 16), dim3(256), 0, st,
                                               x + (size_t)r0 * (size_t)K, q + (size_t)r0 * (size_t)K,
                                               s + (size_t)r0 * Kb, K, Kb, nb);
            if (e != hipSuccess)
                return e;
            if (rows > M - r0)
                break;
        }
        return hipSuccess;
    }
    const unsigned tiles = ((unsigned)M + 127) / 128 * Kb;   // below 2^31
    for (unsigned first = 0; first < tiles; first += 1u << 23) {
        const hipError_t e = launch_kernel(k_f8_quantize_tiles<T>, dim3(std::min(tiles - first, 1u << 23)),
                                           dim3(256), 0, st, x, q, s, M, K, (int)Kb, (int)first);
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

hipError_t launch_f8_quantize(const float *x, uint8_t *q, float *s, int M, int K, int block_rows,
                              hipStream_t st)
{
    return launch_quantize_t<float>(x, q, s, M, K, block_rows, st);
}

hipError_t launch_f8_quantize_bf16(const uint16_t *x, uint8_t *q, float *s, int M, int K,
                                   int block_rows, hipStream_t st)
{
    return launch_quantize_t<uint16_t>(x, q, s, M, K, block_rows, st);
}

// ---------------------------------------------------------------------------
// Decode: out = code * s, one rounding. A thread takes 16 codes.
__global__ __launch_bounds__(256) void k_f8_dequant(const uint8_t *__restrict__ q,
                                                   const float *__restrict__ s,
                                                   float *__restrict__ out, int K, int Kb,
                                                   int block_rows, size_t n16)
{
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n16)
        return;
    const size_t e = i * 16, row = e / (size_t)K;
    const int col = (int)(e - row * (size_t)K);   // K % 32 == 0: 16 codes never straddle rows
    const float sc = s[(row / (size_t)block_rows) * (size_t)Kb + (size_t)(col >> 7)];
    const u32x4 c = reinterpret_cast<const u32x4 *>(q)[i];
    f32x4 *o = reinterpret_cast<f32x4 *>(out + e);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[j], false);
        const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[j], true);
        o[j] = (f32x4){lo[0] * sc, lo[1] * sc, hi[0] * sc, hi[1] * sc};
    }
}

hipError_t launch_f8_dequant(const uint8_t *q, const float *s, float *out, int M, int K,
                             int block_rows, hipStream_t st)
{
    const size_t n16 = (size_t)M * (size_t)K / 16, grid = (n16 + 255) / 256;
    if (grid > 0x7fffffffu)
        return hipErrorInvalidValue;
    return launch_kernel(k_f8_dequant, dim3((unsigned)grid), dim3(256), 0, st, q, s, out, K,
                         (int)(((unsigned)K + 127) / 128), block_rows, n16);
}

// ---------------------------------------------------------------------------
// The product. v_mfma_f32_16x16x128_f8f6f4 contracts one whole block of 128
// codes, so per 16 x 16 tile and block one matrix instruction gives the sum
// over the block and one f32 FMA per element adds it, times a_s w_s, to the
// accumulator. The weights are the A operand and the activations the B
// operand: a lane's four results are then four columns of y of one row, one
// activation scale serves a lane's whole tile column, and they are stored
// together.
//
// Rounding: the instruction forms each run of eight products (the bytes a
// lane's dword pair holds) against the largest of the eight, and drops what is
// below 2^-13 of that one's power of two (measured on the card with one large
// and one small product at every distance); the runs are added in f32. Every
// other 8-bit matrix instruction of the card does the same. On N(0, 1) codes
// that is 1.3e-5 of the result's norm, a hundredth of y's rounding to
// bfloat16 (1.7e-3), and the reason y is bfloat16: an f32 result would claim
// bits that the products do not have. (Widening the codes to binary16 first
// would keep them, at half the matrix rate and eight conversions an operand.)
// Blocks are added in f32 in K order.
//
// The K order within a block does not matter as long as both operands agree:
// lane group g = lane / 16 takes bytes [16 g, 16 g + 16) and [64 + 16 g, 80 +
// 16 g) of its row's block, so every 16-byte load is aligned.

struct F8Product {
    const uint8_t *a;
    const float *a_s;
    const uint8_t *w;
    const float *w_s;
    uint16_t *y;
    int M, N, K, Kb, Nb;
};

__device__ __forceinline__ i32x8 join(u32x4 lo, u32x4 hi)
{
    return (i32x8){(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
                   (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

__device__ __forceinline__ f32x4 mfma_block(i32x8 w, i32x8 a)
{
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, zero, 0, 0, 0, 0, 0, 0);
}

// Columns n .. n + 3 of one row of y.
__device__ __forceinline__ void store4(uint16_t *__restrict__ row, int n, int N, f32x4 v)
{
    const bf16x4 b = {(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
    if ((N & 3) == 0) {
        if (n < N)
            *reinterpret_cast<bf16x4 *>(row + n) = b;
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (n + q < N)
                reinterpret_cast<__bf16 *>(row)[n + q] = b[q];
    }
}

constexpr uint32_t kOutOfRange = 0x80000000u;   // past every resource below (each spans at most 2^31 bytes)
constexpr int kRawBuffer = 0x00020000;          // resource word 3: raw, 32-bit data format

// vmcnt(vm) lgkmcnt(0).
constexpr int wait_loads(int vm) { return (vm & 15) | ((vm >> 4) << 14) | 0x70; }

// Few rows: bound by the weights' bytes. A workgroup takes 16 weight rows and up
// to 16 RG activation rows; its NW wavefronts each take a contiguous run of the
// blocks of K and add their partial tiles through LDS at the end. A wavefront
// stages its own blocks in its own LDS by direct loads, whole 128-byte lines of
// eight rows a load, in a ring of NST blocks, and so waits for its own loads
// only (registers would take each row in two half lines, and hold fewer
// bytes in flight). 16-byte pieces are stored at piece ^ (row % 8): the eight
// rows of an LDS read lie in different banks. The rows' scales come four blocks
// at a time, the weights' scales 64 at a time, one a lane.
template <int RG_, int NW_, int NST_>
struct RowsShape {
    static constexpr int RG = RG_, NW = NW_, NST = NST_;
    static constexpr int kThreads = 64 * NW;
    static constexpr int kLoads = 2 + 2 * RG;                 // of a block
    static constexpr int kStage = 128 + RG * 128;             // 16-byte words of a block: weights, activations
    static_assert(NST >= 2 && (NST - 2) * kLoads < 64 && NST <= 5, "vmcnt counts to 63; scales land a chunk ahead");
};

template <class S>
struct RowsLds {
    union {
        struct {
            u32x4 blk[S::NW][S::NST][S::kStage];
            float s[S::NW][2][S::RG * 64];                    // [row / 16][block % 4][row % 16]
        };
        f32x4 red[S::RG][S::NW][64];
    };
};

// Weight rows n0 .. n0 + 15 of (w, w_s) times the rows at(0) .. at(16 RG - 1)
// (activation row and row of y; -1 for none).
template <class S, class At>
__device__ __forceinline__ void rows_tile(const F8Product &p, const uint8_t *__restrict__ w,
                                          const float *__restrict__ w_s, uint32_t a_rows, int n0,
                                          At at, RowsLds<S> &lds)
{
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int li = lane & 15, g = lane >> 4;
    const int wrows = min(16, p.N - n0);
    const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(w + (size_t)n0 * (size_t)p.K), (short)0, (int)((uint32_t)wrows * (uint32_t)p.K), kRawBuffer);
    const __amdgpu_buffer_rsrc_t ar = __builtin_amdgcn_make_buffer_rsrc(
        (void *)p.a, (short)0, (int)(a_rows * (uint32_t)p.K), kRawBuffer);
    const __amdgpu_buffer_rsrc_t sr = __builtin_amdgcn_make_buffer_rsrc(
        (void *)p.a_s, (short)0, (int)(a_rows * (uint32_t)p.Kb * 4u), kRawBuffer);
    const int per = (p.Kb + S::NW - 1) / S::NW;
    const int b0 = wave * per, b1 = min(b0 + per, p.Kb);

    // Load j: rows 8 j + lane / 8, piece (lane % 8) ^ (row % 8).
    const int lr = lane >> 3, piece = ((lane ^ lr) & 7) * 16;
    uint32_t wo[2], ao[2 * S::RG], so[S::RG];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int r = 8 * j + lr;
        wo[j] = r < wrows ? (uint32_t)r * (uint32_t)p.K + (uint32_t)piece : kOutOfRange;
    }
#pragma unroll
    for (int j = 0; j < 2 * S::RG; ++j) {
        const int x = at(8 * j + lr).x;
        ao[j] = x >= 0 ? (uint32_t)x * (uint32_t)p.K + (uint32_t)piece : kOutOfRange;
    }
#pragma unroll
    for (int r = 0; r < S::RG; ++r) {
        const int x = at(16 * r + li).x;
        so[r] = x >= 0 ? ((uint32_t)x * (uint32_t)p.Kb + (uint32_t)g) * 4u : kOutOfRange;
    }
    auto issue = [&](int b) __attribute__((always_inline)) {
        u32x4 *to = lds.blk[wave][(unsigned)(b - b0) % S::NST];
        // Pieces past K, and blocks past the run, read as zero.
        const bool in = b < b1 && piece < p.K - b * 128;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            load16_to_lds(wr, to + j * 64, in ? wo[j] : kOutOfRange, b * 128);
#pragma unroll
        for (int j = 0; j < 2 * S::RG; ++j)
            load16_to_lds(ar, to + 128 + j * 64, in ? ao[j] : kOutOfRange, b * 128);
    };
    auto issue_scales = [&](int c) __attribute__((always_inline)) {   // blocks b0 + 4 c ..
        const bool in = b0 + 4 * c + g < b1;
#pragma unroll
        for (int r = 0; r < S::RG; ++r)
            load4_to_lds(sr, lds.s[wave][c & 1] + r * 64, in ? so[r] : kOutOfRange, (b0 + 4 * c) * 4);
    };

    f32x4 acc[S::RG];
#pragma unroll
    for (int r = 0; r < S::RG; ++r)
        acc[r] = (f32x4){0.f, 0.f, 0.f, 0.f};
    const int o0 = li * 8 + (g ^ (li & 7)), o1 = li * 8 + ((4 + g) ^ (li & 7));
    if (b0 < b1) {
        float ws64 = w_s[min(b0 + lane, p.Kb - 1)];
        issue_scales(0);
#pragma unroll
        for (int d = 0; d < S::NST - 1; ++d)
            issue(b0 + d);
        for (int b = b0; b < b1; ++b) {
            const int i = b - b0;
            if ((i & 63) == 0 && i > 0)
                ws64 = w_s[min(b + lane, p.Kb - 1)];
            const float ws = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ws64), i & 63));
            // This block (and its scales, which are older) has landed, and the
            // block before it is in registers: its place takes block b + NST - 1.
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(wait_loads((S::NST - 2) * S::kLoads));
            asm volatile("" ::: "memory");
            if ((i & 3) == 0)
                issue_scales((i >> 2) + 1);
            issue(b + S::NST - 1);
            asm volatile("" ::: "memory");
            const u32x4 *from = lds.blk[wave][(unsigned)i % S::NST];
            const float *sp = lds.s[wave][(i >> 2) & 1] + (i & 3) * 16 + li;
            const i32x8 wf = join(from[o0], from[o1]);
#pragma unroll
            for (int r = 0; r < S::RG; ++r) {
                const i32x8 af = join(from[128 + r * 128 + o0], from[128 + r * 128 + o1]);
                const f32x4 c = mfma_block(wf, af);
                const float s = sp[r * 64] * ws;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    acc[r][q] = fmaf(s, c[q], acc[r][q]);
            }
        }
    }
    // Partial tiles; wavefront r mod NW adds tile r's in wavefront order.
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(wait_loads(0));
    __syncthreads();
#pragma unroll
    for (int r = 0; r < S::RG; ++r)
        lds.red[r][wave][lane] = acc[r];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < S::RG; ++r) {
        const int to = at(16 * r + li).y;
        if (r % S::NW != wave || to < 0)
            continue;
        f32x4 v = lds.red[r][0][lane];
#pragma unroll
        for (int s = 1; s < S::NW; ++s)
            v += lds.red[r][s][lane];
        store4(p.y + (size_t)to * (size_t)p.N, n0 + 4 * g, p.N, v);
    }
}

// Workgroup (x, t): weight rows 16 x .., activation rows 16 RG t ...
template <class S>
__global__ __launch_bounds__(S::kThreads) void k_f8_rows(F8Product p, int first)
{
    __shared__ RowsLds<S> lds;
    const int x = first + (int)blockIdx.x;
    const int m0 = blockIdx.y * (16 * S::RG), rows = min(16 * S::RG, p.M - m0);
    p.a += (size_t)m0 * (size_t)p.K;
    p.a_s += (size_t)m0 * (size_t)p.Kb;
    auto at = [&](int r) __attribute__((always_inline)) {
        return r < rows ? int2{r, m0 + r} : int2{-1, -1};
    };
    rows_tile<S>(p, p.w, p.w_s + (size_t)(x >> 3) * (size_t)p.Kb, (uint32_t)rows, x * 16, at, lds);
}

// The same over groups: workgroup (x, e) takes 16 weight rows of group e past
// the group's rows, 16 RG at a time.
template <class S>
__global__ __launch_bounds__(S::kThreads) void k_f8_rows_grouped(F8Product p, Groups gr, int first)
{
    __shared__ RowsLds<S> lds;
    const int e = blockIdx.y, x = first + (int)blockIdx.x;
    int lo, hi;
    group_bounds(gr, e, lo, hi);
    const uint8_t *w = p.w + (size_t)e * (size_t)p.N * (size_t)p.K;
    const float *w_s = p.w_s + ((size_t)e * (size_t)p.Nb + (size_t)(x >> 3)) * (size_t)p.Kb;
    const uint32_t a_rows = (uint32_t)((gr.M - 1) / gr.share + 1);
    for (; lo < hi; lo += 16 * S::RG) {
        auto at = [&](int r) __attribute__((always_inline)) {
            const int y = lo + r < hi ? group_row(gr, lo + r) : -1;
            return int2{y < 0 ? -1 : y / gr.share, y};
        };
        rows_tile<S>(p, w, w_s, a_rows, x * 16, at, lds);
        __syncthreads();   // the partial tiles are read before the next rows' loads
    }
}

using Rows1 = RowsShape<1, 8, 4>;
using Rows2 = RowsShape<2, 8, 3>;
using Rows3 = RowsShape<3, 4, 4>;
using Rows4 = RowsShape<4, 4, 3>;

// More rows: bound by the matrix instructions. A workgroup of eight wavefronts
// computes BN x BM of y^T, WN x WM x KS wavefronts of TN x TM tiles each. Per
// step (KS blocks of K, each taken by the WN x WM wavefronts of one half) it
// stages both operands in LDS by direct loads, in a ring of NS stages. With few
// tiles a step is as long as its chain of latencies (barrier, LDS, matrix
// instruction, FMA: 0.3 us), so the small shapes take two blocks a step and add
// the halves at the end (256 x 4096 x 4096 in 64 x 64 tiles: 13.6 us with one
// block a step, 11.4 with two); the larger shapes need the LDS for the ring.
// 16-byte pieces of a row's 128 bytes are stored at piece ^ (row % 8), so that
// the 8 rows that an LDS read serves at a time lie in different banks (the
// lanes' global addresses carry the permutation; the LDS side of a direct load
// is contiguous). The activation scales of eight blocks are staged at a time:
// loaded step by step, a scale of each of 64 rows a load, they took as many
// cache lines as both operands twice over.
template <int WN_, int WM_, int TN_, int TM_, int NS_, int KS_ = 1>
struct TileShape {
    static constexpr int WN = WN_, WM = WM_, TN = TN_, TM = TM_, NS = NS_, KS = KS_;
    static constexpr int BN = WN * TN * 16, BM = WM * TM * 16;
    static constexpr int kThreads = 64 * WN * WM * KS;
    static constexpr int kWLoads = KS * BN * 8 / kThreads, kALoads = KS * BM * 8 / kThreads;
    static constexpr int kLoads = kWLoads + kALoads;       // of every wavefront and step
    static constexpr int kSLoads = BM * 8 / kThreads;      // of a chunk of scales
    static constexpr int kInFlight = (NS - 2) * kLoads;    // younger than the stage that a turn waits for
    // Matrix instructions of a step and wavefront; the one before which the
    // stages change over, with one column of tiles to go.
    static constexpr int kTiles = TN * TM, kTurn = (TM - 1) * TN;
    // Slots of a step's loads: behind the matrix instructions from the turn to
    // the end of the step, then of the next step's first kSpread (which end
    // before its turn; with two stages the loads must land by then, so they
    // stop earlier). kTailLoads of the loads fall before the step's end.
    static constexpr int kSpread = NS == 2 ? TN : kTurn, kSlots = TN + kSpread;
    static constexpr int kTailLoads = TN * kLoads / kSlots;
    static constexpr int kRowBytes = BN * 2 + 16;          // of a row of y in LDS
    static constexpr int kChunk = 8 / KS;                  // steps of a chunk of scales
    static_assert(BN * 8 % kThreads == 0 && BM * 8 % kThreads == 0 && BM % 64 == 0 && BM <= kThreads, "whole loads");
    static_assert((KS == 1 || KS == 2) && NS - 2 < kChunk - 1, "scales land a chunk ahead");
    static_assert(TN * 16 <= 128 && 128 % (TN * 16) == 0, "a wavefront's columns share a weight scale");
    static_assert(TM % 2 == 0, "activation operands alternate between two registers");
    static_assert(NS >= 2 && kInFlight < 64, "vmcnt counts to 63");
};

template <class S>
struct TileLds {
    union {
        struct {
            u32x4 w[S::NS][S::KS * S::BN * 8];
            u32x4 a[S::NS][S::KS * S::BM * 8];
        };
        f32x4 red[S::KS == 1 ? 1 : S::WN * S::WM * S::kTiles][64];
        uint8_t y[S::BM * S::kRowBytes];
    };
    float s[2][S::BM * 8];   // of eight steps: [row / 8][step][row % 8]
    int row[S::BM];
};

// Wait until at most VM of the wavefront's loads are in flight and its LDS
// operations are done, then meet the others.
template <int VM>
__device__ __forceinline__ void wait_and_meet()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(wait_loads(VM));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Tiles to XCDs (workgroup index mod 8): XCD (x, y) of an nx x ny grid takes a
// rectangle of rn x rm tiles, walked in strips of eight row tiles, so that the
// workgroups that run on it together share both operands in its L2.
struct TileOrder {
    int tn, tm;   // tiles
    int nx, rn, rm;
};

__device__ __forceinline__ bool tile_of(const TileOrder &o, int L, int &nt, int &mt)
{
    const int x = L & 7, i = L >> 3;
    const int xn = x % o.nx, xm = x / o.nx;
    const int strip = i / (8 * o.rn), h = min(8, o.rm - 8 * strip), r = i - strip * 8 * o.rn;
    nt = xn * o.rn + r / h;
    mt = xm * o.rm + 8 * strip + r % h;
    return nt < o.tn && mt < o.tm;
}

template <class S, bool GROUPED>
__global__ __launch_bounds__(S::kThreads) void k_f8_tile(F8Product p, Groups gr, TileOrder order, int first)
{
    __shared__ TileLds<S> lds;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int mt, nt, rows;
    const uint8_t *w = p.w;
    const float *w_s = p.w_s;
    if constexpr (GROUPED) {
        const GroupTile g = find_group_tile(gr, xcd_runs(first + (int)blockIdx.x), S::BM, order.tn);
        if (g.e < 0)
            return;
        mt = g.mt, nt = g.nt;
        const int lo = g.lo + mt * S::BM;
        rows = min(S::BM, g.hi - lo);
        w += (size_t)g.e * (size_t)p.N * (size_t)p.K;
        w_s += (size_t)g.e * (size_t)p.Nb * (size_t)p.Kb;
        if (tid < S::BM)
            lds.row[tid] = tid < rows ? group_row(gr, lo + tid) : -1;
        __syncthreads();
    } else {
        if (!tile_of(order, first + (int)blockIdx.x, nt, mt))
            return;
        rows = min(S::BM, p.M - mt * S::BM);
    }
    const int n0 = nt * S::BN, m0 = mt * S::BM;
    const int li = lane & 15, g = lane >> 4;
    const int wn = wave % S::WN, wm = wave / S::WN % S::WM, ks = wave / (S::WN * S::WM);

    // Resources: this tile's weight rows; its activation rows and scales, or
    // (grouped) all of them.
    const int wrows = min(S::BN, p.N - n0);
    const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(w + (size_t)n0 * (size_t)p.K), (short)0, (int)((uint32_t)wrows * (uint32_t)p.K), kRawBuffer);
    const size_t am0 = GROUPED ? 0 : (size_t)m0;
    const uint32_t arows = GROUPED ? (uint32_t)((gr.M - 1) / gr.share + 1) : (uint32_t)rows;
    const __amdgpu_buffer_rsrc_t ar = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(p.a + am0 * (size_t)p.K), (short)0, (int)(arows * (uint32_t)p.K), kRawBuffer);
    const __amdgpu_buffer_rsrc_t sr = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(p.a_s + am0 * (size_t)p.Kb), (short)0, (int)(arows * (uint32_t)p.Kb * 4u), kRawBuffer);

    // Activation row of the tile's row r, or -1.
    auto a_row = [&](int r) __attribute__((always_inline)) {
        if constexpr (GROUPED) {
            const int x = lds.row[r];
            return x < 0 ? -1 : x / gr.share;
        } else {
            return r < rows ? r : -1;
        }
    };
    // Offsets of this lane's pieces in step 0. Load j of a wavefront covers rows
    // of one residue mod 8, so its piece of the row is the same in all of them.
    uint32_t wo[S::kWLoads], ao[S::kALoads], so[S::kSLoads];
    const int piece = ((tid ^ (tid >> 3)) & 7) * 16;
    static_assert(S::kThreads % 64 == 0, "rows of a load are equal mod 8");
#pragma unroll
    for (int j = 0; j < S::kWLoads; ++j) {
        const int r = ((j * S::kThreads + tid) >> 3) % S::BN;
        wo[j] = r < wrows ? (uint32_t)r * (uint32_t)p.K + (uint32_t)piece : kOutOfRange;
    }
#pragma unroll
    for (int j = 0; j < S::kALoads; ++j) {
        const int x = a_row(((j * S::kThreads + tid) >> 3) % S::BM);
        ao[j] = x >= 0 ? (uint32_t)x * (uint32_t)p.K + (uint32_t)piece : kOutOfRange;
    }
#pragma unroll
    for (int j = 0; j < S::kSLoads; ++j) {
        const int x = a_row((j * S::kThreads + tid) / 64 * 8 + (lane & 7));
        so[j] = x >= 0 ? ((uint32_t)x * (uint32_t)p.Kb + (uint32_t)(lane >> 3)) * 4u : kOutOfRange;
    }
    const int steps = (p.Kb + S::KS - 1) / S::KS;
    // Block of a step that load j takes a part of.
    auto w_block = [](int j) { return j * S::kThreads / (S::BN * 8); };
    auto a_block = [](int j) { return j * S::kThreads / (S::BM * 8); };
    // Called before a step's loads, in order of the steps: in a short last step
    // the pieces past K, and after it everything, move out of range, where they
    // read as zero. No earlier step needs the offsets again.
    auto trim = [&](int step) __attribute__((always_inline)) {
        const int left = p.K - step * (S::KS * 128);
        if (left >= S::KS * 128)
            return;
#pragma unroll
        for (int j = 0; j < S::kWLoads; ++j)
            wo[j] = piece >= left - w_block(j) * 128 ? kOutOfRange : wo[j];
#pragma unroll
        for (int j = 0; j < S::kALoads; ++j)
            ao[j] = piece >= left - a_block(j) * 128 ? kOutOfRange : ao[j];
    };
    // The scales of blocks 8 c .. 8 c + 7; those past the last block read as zero.
    auto issue_scales = [&](int c) __attribute__((always_inline)) {
        const bool in = 8 * c + (lane >> 3) < p.Kb;
#pragma unroll
        for (int j = 0; j < S::kSLoads; ++j)
            load4_to_lds(sr, lds.s[c & 1] + j * S::kThreads + wave * 64, in ? so[j] : kOutOfRange, c * 32);
    };
    // Load l of a step into its stage st.
    auto issue = [&](int step, int st, int l) __attribute__((always_inline)) {
        if (l < S::kWLoads)
            load16_to_lds(wr, lds.w[st] + l * S::kThreads + wave * 64, wo[l],
                         (step * S::KS + w_block(l)) * 128);
        else
            load16_to_lds(ar, lds.a[st] + (l - S::kWLoads) * S::kThreads + wave * 64, ao[l - S::kWLoads],
                          (step * S::KS + a_block(l - S::kWLoads)) * 128);
    };

    f32x4 acc[S::TN][S::TM];
#pragma unroll
    for (int i = 0; i < S::TN; ++i)
#pragma unroll
        for (int j = 0; j < S::TM; ++j)
            acc[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
    const int nb = min((n0 + wn * (S::TN * 16)) >> 7, p.Nb - 1);
    // Uniform over the wavefront: read through the scalar cache, so that waiting
    // for it does not wait for the vector loads in flight.
    const __attribute__((address_space(4))) int *wsp =
        (const __attribute__((address_space(4))) int *)(uintptr_t)(w_s + (size_t)nb * (size_t)p.Kb);

    // Operand of a 16-row tile in LDS: pieces g and 4 + g of row li.
    const int o0 = li * 8 + (g ^ (li & 7)), o1 = li * 8 + ((4 + g) ^ (li & 7));
    auto operand = [&](const u32x4 *base) __attribute__((always_inline)) { return join(base[o0], base[o1]); };
    auto w_operand = [&](int st, int i) __attribute__((always_inline)) {
        return operand(lds.w[st] + (ks * (S::BN / 16) + wn * S::TN + i) * 128);
    };
    auto a_operand = [&](int st, int j) __attribute__((always_inline)) {
        return operand(lds.a[st] + (ks * (S::BM / 16) + wm * S::TM + j) * 128);
    };

    auto read_scales = [&](int step, float (&to)[S::TM]) __attribute__((always_inline)) {
        const int b = step * S::KS + ks;
        const float *base = lds.s[(b >> 3) & 1] + (wm * S::TM * 2 + (li >> 3)) * 64 + (b & 7) * 8 + (li & 7);
#pragma unroll
        for (int x = 0; x < S::TM; ++x)
            to[x] = base[x * 128];
    };

    // The pipeline. Step s multiplies stage s mod NS. Its weight operands, its
    // first activation operand and its scales are in registers when it begins, so
    // no step begins by waiting for LDS. At kTurn every wavefront has read the
    // last of the stage (the wait and the barrier) and the next stage has landed:
    // the step's last column of tiles runs from registers while each weight
    // operand that it has used is read again from the next stage, and the loads
    // of step s + NS begin to fill the stage just left; they are spread into the
    // next step, since a burst of them from every wavefront at once stalls the
    // issue of all. Tile t's FMAs follow matrix instruction t + kLag, when its
    // result is ready. The group barriers keep that order; the empty asm keeps
    // the FMAs where they are written. The last kLag tiles' FMAs of a step run in
    // the next one (kCarry), which then begins with matrix instructions; not in
    // the large form, whose registers are all taken, and where they are a
    // sixteenth of the tiles.
    constexpr int kLag = 2, kRing = 4;
    constexpr bool kCarry = S::kTiles < 32;
    static_assert(S::kTiles % kRing == 0 && S::TN >= kLag, "results of two steps do not meet");
    i32x8 wf[S::TN], af[2];
    f32x4 c[kRing];
    float as[S::TM], sc[S::TM], sc_last = 0.0f;
    int ws_next;
#pragma unroll
    for (int i = 0; i < kRing; ++i)
        c[i] = (f32x4){0.f, 0.f, 0.f, 0.f};
    auto add_tile = [&](auto u_c, float s) __attribute__((always_inline)) {
        constexpr int u = decltype(u_c)::value, i = u % S::TN, j = u / S::TN;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            acc[i][j][q] = fmaf(s, c[u % kRing][q], acc[i][j][q]);
        asm volatile("" : "+v"(acc[i][j]));
    };
    auto run_step = [&](auto st_c, int step) __attribute__((always_inline)) {
        constexpr int P = decltype(st_c)::value, Q = (P + 1) % S::NS;
        const float ws = __int_as_float(ws_next);
        sc_last = sc[S::TM - 1];
#pragma unroll
        for (int j = 0; j < S::TM; ++j)
            sc[j] = as[j] * ws;
        // Chunk step / 8 - 1 was last read before the previous step's end, so
        // the next chunk may take its place; it lands within eight steps, older
        // by then than any load that a turn leaves in flight.
        if (step % S::kChunk == 0)
            issue_scales(step / S::kChunk + 1);
        __builtin_amdgcn_sched_barrier(0);
        unroll<S::kTiles + (kCarry ? 0 : kLag)>([&](auto t_c) __attribute__((always_inline)) {
            constexpr int t = decltype(t_c)::value, i = t % S::TN, j = t / S::TN;
            if constexpr (t == S::kTurn) {
                __builtin_amdgcn_sched_barrier(0);
                wait_and_meet<S::kInFlight>();
                asm volatile("" : "+s"(ws_next));
                trim(step + S::NS);
                __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (t < S::kTiles) {
                c[t % kRing] = mfma_block(wf[i], af[j & 1]);
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                if constexpr (i == 0 && j + 1 < S::TM) {
                    af[(j + 1) & 1] = a_operand(P, j + 1);
                    __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
                }
                if constexpr (t == S::kTurn - S::TN) {
                    // Here no LDS result is waited for before the turn, so the
                    // scalar load in flight makes no such wait longer.
                    __builtin_amdgcn_sched_barrier(0);
                    ws_next = wsp[min((step + 1) * S::KS + ks, p.Kb - 1)];
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            if constexpr (t >= S::kTurn && t < S::kTiles) {
                wf[i] = w_operand(Q, i);
                __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
                if constexpr (i == 0) {   // the last column reads af[1]
                    af[0] = a_operand(Q, 0);
                    read_scales(step + 1, as);
                }
            }
            if constexpr (t < S::kSpread || (t >= S::kTurn && t < S::kTiles)) {
                constexpr bool tail = t >= S::kTurn;
                constexpr int u = tail ? i : S::TN + t;
                constexpr int l0 = u * S::kLoads / S::kSlots, l1 = (u + 1) * S::kLoads / S::kSlots;
                unroll<l1 - l0>([&](auto l) __attribute__((always_inline)) {
                    issue(step + S::NS - (tail ? 0 : 1), tail ? P : (P + S::NS - 1) % S::NS, l0 + l.value);
                    __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
                });
            }
            if constexpr (t >= kLag || kCarry) {
                if constexpr (t >= kLag)
                    add_tile(std::integral_constant<int, t - kLag>{}, sc[(t - kLag) / S::TN]);
                else
                    add_tile(std::integral_constant<int, S::kTiles - kLag + t>{}, sc_last);
                __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
            }
        });
        __builtin_amdgcn_sched_barrier(0);
    };

    issue_scales(0);
#pragma unroll
    for (int s = 0; s < S::NS; ++s) {
        trim(s);
#pragma unroll
        for (int l = 0; l < (s < S::NS - 1 ? S::kLoads : S::kTailLoads); ++l)
            issue(s, s, l);
    }
    ws_next = wsp[min(ks, p.Kb - 1)];
    wait_and_meet<S::kInFlight + S::kTailLoads>();
#pragma unroll
    for (int i = 0; i < S::TN; ++i)
        wf[i] = w_operand(0, i);
    af[0] = a_operand(0, 0);
    read_scales(0, as);
#pragma unroll
    for (int x = 0; x < S::TM; ++x)
        sc[x] = 0.0f;
    for (int step = 0; step < steps; step += S::NS)
        unroll<S::NS>([&](auto s) __attribute__((always_inline)) {
            if (step + s.value < steps)
                run_step(s, step + s.value);
        });
    if constexpr (kCarry)
        unroll<kLag>([&](auto t) __attribute__((always_inline)) {
            add_tile(std::integral_constant<int, S::kTiles - kLag + t.value>{}, sc[S::TM - 1]);
        });
    wait_and_meet<0>();   // no load is on its way into the LDS that the epilogue uses
    if constexpr (S::KS == 2) {
        // The second half of the wavefronts hands its sums to the first.
        f32x4 (*red)[64] = lds.red + wave % (S::WN * S::WM) * S::kTiles;
        if (ks != 0) {
#pragma unroll
            for (int t = 0; t < S::kTiles; ++t)
                red[t][lane] = acc[t % S::TN][t / S::TN];
        }
        __syncthreads();
        if (ks == 0) {
#pragma unroll
            for (int t = 0; t < S::kTiles; ++t)
                acc[t % S::TN][t / S::TN] += red[t][lane];
        }
        __syncthreads();
    }

    // y: through LDS, so that whole rows of the tile leave as 16-byte stores of
    // consecutive lanes (where the rows of y allow them).
    auto y_row = [&](int r) __attribute__((always_inline)) {
        if constexpr (GROUPED)
            return lds.row[r];
        else
            return r < rows ? m0 + r : -1;
    };
    if ((p.N & 7) == 0) {
#pragma unroll
        for (int j = 0; j < S::TM; ++j) {
            if (ks != 0)
                break;
            uint8_t *row = lds.y + ((wm * S::TM + j) * 16 + li) * S::kRowBytes + (wn * (S::TN * 16) + 4 * g) * 2;
#pragma unroll
            for (int i = 0; i < S::TN; ++i) {
                const f32x4 v = acc[i][j];
                *reinterpret_cast<bf16x4 *>(row + i * 32) = (bf16x4){(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
            }
        }
        __syncthreads();
        constexpr int kLanes = S::BN / 8, kRowsAtOnce = S::kThreads / kLanes;   // 16-byte pieces of a row
        const int n = n0 + tid % kLanes * 8;
        for (int r = tid / kLanes; r < S::BM; r += kRowsAtOnce) {
            const int to = y_row(r);
            if (to >= 0 && n < p.N)
                *reinterpret_cast<u32x4 *>(p.y + (size_t)to * (size_t)p.N + n) =
                    *reinterpret_cast<const u32x4 *>(lds.y + r * S::kRowBytes + tid % kLanes * 16);
        }
    } else if (ks == 0) {
#pragma unroll
        for (int j = 0; j < S::TM; ++j) {
            const int to = y_row((wm * S::TM + j) * 16 + li);
            if (to < 0)
                continue;
            uint16_t *yp = p.y + (size_t)to * (size_t)p.N;
#pragma unroll
            for (int i = 0; i < S::TN; ++i)
                store4(yp, n0 + wn * (S::TN * 16) + i * 16 + 4 * g, p.N, acc[i][j]);
        }
    }
}

using TileQuarter = TileShape<2, 2, 2, 2, 4, 2>;   // 64 columns x 64 rows
using TileHalf = TileShape<2, 2, 4, 2, 3, 2>;      // 128 x 64
using TileSmall = TileShape<2, 4, 4, 2, 4>;        // 128 x 128
using TileWide = TileShape<4, 2, 4, 4, 3>;         // 256 x 128
using TileLarge = TileShape<2, 4, 8, 4, 2>;        // 256 x 256

template <class S>
static hipError_t launch_tiles(const F8Product &p, hipStream_t st)
{
    static_assert(sizeof(TileLds<S>) <= 160 * 1024, "the ring fits in LDS");
    const long long tm = ((long long)p.M + S::BM - 1) / S::BM, tn = ((long long)p.N + S::BN - 1) / S::BN;
    // The split of the tiles over the XCDs that leaves the fewest slots empty,
    // and of those the one whose rectangle is nearest a square.
    TileOrder o = {(int)tn, (int)tm, 0, 0, 0};
    long long best = 0;
    for (int nx = 1; nx <= 8; nx *= 2) {
        const long long rn = (tn + nx - 1) / nx, rm = (tm + 8 / nx - 1) / (8 / nx);
        if (!best || rn * rm < best || (rn * rm == best && rn + rm < (long long)o.rn + o.rm))
            best = rn * rm, o.nx = nx, o.rn = (int)rn, o.rm = (int)rm;
    }
    if (best * 8 > 0x7fffffffLL)
        return hipErrorInvalidValue;
    return launch_parts(k_f8_tile<S, false>, best * 8, 1, S::kThreads, st, p,
                        Groups{nullptr, nullptr, 0, 0, 1, 0}, o);
}

template <class S>
static hipError_t launch_rows(const F8Product &p, hipStream_t st)
{
    static_assert(sizeof(RowsLds<S>) <= 160 * 1024, "the rings fit in LDS");
    return launch_parts(k_f8_rows<S>, ((long long)p.N + 15) / 16,
                        (unsigned)((p.M + 16LL * S::RG - 1) / (16 * S::RG)), S::kThreads, st, p);
}

template <class S>
static hipError_t launch_rows_grouped(const F8Product &p, const Groups &gr, hipStream_t st)
{
    return launch_parts(k_f8_rows_grouped<S>, ((long long)p.N + 15) / 16, (unsigned)gr.G, S::kThreads, st, p, gr);
}

// f8_forms.h prices the tiles by their sides.
template <class S>
constexpr bool sides(q4v::F8Form f) { return q4v::kF8Tiles[f - q4v::kF8Quarter].bn == S::BN && q4v::kF8Tiles[f - q4v::kF8Quarter].bm == S::BM; }
static_assert(sides<TileQuarter>(q4v::kF8Quarter) && sides<TileHalf>(q4v::kF8Half) && sides<TileSmall>(q4v::kF8Small) &&
                  sides<TileWide>(q4v::kF8Wide) && sides<TileLarge>(q4v::kF8Large), "one list of sides");

hipError_t launch_f8_gemm(const uint8_t *a, const float *a_s, const uint8_t *w, const float *w_s,
                          uint16_t *y, int M, int N, int K, hipStream_t st)
{
    const F8Product p = {a, a_s, w, w_s, y, M, N, K, (K + 127) / 128, (int)(((long long)N + 127) / 128)};
    const q4v::F8Choice c = q4v::f8_form(M, N);
    switch (c.form) {
    case q4v::kF8Rows:
        return c.rg == 1 ? launch_rows<Rows1>(p, st) : c.rg == 2 ? launch_rows<Rows2>(p, st)
             : c.rg == 3 ? launch_rows<Rows3>(p, st) : launch_rows<Rows4>(p, st);
    case q4v::kF8Quarter: return launch_tiles<TileQuarter>(p, st);
    case q4v::kF8Half: return launch_tiles<TileHalf>(p, st);
    case q4v::kF8Small: return launch_tiles<TileSmall>(p, st);
    case q4v::kF8Wide: return launch_tiles<TileWide>(p, st);
    default: return launch_tiles<TileLarge>(p, st);
    }
}

template <class S>
static hipError_t launch_grouped_tiles(const F8Product &p, const Groups &gr, hipStream_t st)
{
    const long long tn = ((long long)p.N + S::BN - 1) / S::BN;
    const long long grid = group_grid(gr.G, gr.M, S::BM, tn);
    if (grid > kMaxGroupTiles)
        return hipErrorInvalidValue;
    return launch_parts(k_f8_tile<S, true>, grid, 1, S::kThreads, st, p, gr, TileOrder{(int)tn, 0, 0, 0, 0});
}

hipError_t launch_f8_gemm_grouped(const uint8_t *a, const float *a_s, const uint8_t *w,
                                  const float *w_s, const int *offsets, const int *order, int share,
                                  uint16_t *y, int G, int M, int N, int K, hipStream_t st)
{
    const F8Product p = {a, a_s, w, w_s, y, M, N, K, (K + 127) / 128, (int)(((long long)N + 127) / 128)};
    const Groups gr = {offsets, order, G, M, share, 0};
    const q4v::F8Choice c = q4v::f8_form_grouped(G, M, N);
    switch (c.form) {
    case q4v::kF8Rows:
        return c.rg == 1 ? launch_rows_grouped<Rows1>(p, gr, st) : c.rg == 2 ? launch_rows_grouped<Rows2>(p, gr, st)
             : launch_rows_grouped<Rows4>(p, gr, st);
    case q4v::kF8Quarter: return launch_grouped_tiles<TileQuarter>(p, gr, st);
    case q4v::kF8Half: return launch_grouped_tiles<TileHalf>(p, gr, st);
    case q4v::kF8Small: return launch_grouped_tiles<TileSmall>(p, gr, st);
    case q4v::kF8Wide: return launch_grouped_tiles<TileWide>(p, gr, st);
    default: return launch_grouped_tiles<TileLarge>(p, gr, st);
    }
}

}  // namespace q4k
