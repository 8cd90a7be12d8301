// Prefill-shaped block-quantized x f32 product, y[m, n] = sum_k a[m, k] w[n, k]
// for any M, tiled through LDS onto gfx950 matrix cores, for Q4_0 and Q8_0
// weight streams.
//
// Operation: docs.rs fuel-dispatch, "quantized (GGML) kernel contracts",
// section matmul_q4_0_tiled (M > 1, 2 M N K flops, the weight streamed once
// per column block and reused across the rows of a tile), with the blocks of
// sections dequant_q4_0 and dequant_q8_0 (the quantized-matmul binding picks
// either by quant type).
//
// Range: every activation row m is first scaled by a power of two 2^p_m
// (k_row_exp_f32) that puts its largest magnitude in [2^14, 2^15), so any
// finite f32 row fits the binary16 terms below; each result row is scaled back
// by 2^-p_m (exact unless it lands among the f32 subnormals).
//
// Summation order (worst case, u = 2^-24): the two-term split is within 2^-22
// (4u) of each scaled activation; an MFMA block partial adds the lo products
// (each at most 2^-11 of its hi product) first and the hi products onto them,
// about 32u; the scale FMAs d * C + acc then add at most kMaxChain block
// partials in sequence per accumulator, the K groups' tiles are added once,
// and longer K is cut into segments (separate launches, each adding its part
// into y). With S segments the error is at most (36 + kMaxChain + S) u of
// sum |a w|: 150u < 1e-5 for K up to 14336, and below 1e-5 while S <= 19.
//
// General kernel (k_gemm_any, any K % 32 == 0)
// -------------------------------------------
// * A 256-thread workgroup computes a 128 x 128 tile of y; its four wavefronts
//   each own a 64 x 64 quadrant as 4 x 4 tiles of v_mfma_f32_16x16x32_f16.
//   K advances one block (32 elements) per step.
// * Per step the workgroup stages, in LDS, the activation slab a[128 x 32] as
//   binary16 hi = f16(a) and lo = f16((a - hi) * 2^11), and the weight slab as
//   the exact binary16 weight codes plus the same values times 2^-11, with
//   the f32 scales d of the 128 weight rows. For a in [2^e, 2^(e+1)) the
//   residual a - hi is at most 2^(e-11), so lo is at most 2^e <= |a|: no
//   overflow once the row is scaled below 2^15, and lo stays a normal binary16
//   unless the residual is below 2^-25. The matching 2^-11 on the weights
//   (exact) makes hi * c + lo * c 2^-11 equal a c to about 2^-22 relative, so
//   both land in one MFMA chain.
// * Every 16 x 16 tile's block partial is scaled by its column's d into an f32
//   accumulator (d * C + acc): block partial -> scale -> sum of blocks.
// * Two LDS stages with the next step's global loads issued before the current
//   step's MFMAs; one barrier per step.
// * Tiles are renumbered so that each of the chip's 8 XCDs (which receive
//   workgroups round-robin) works on a contiguous run of tiles sharing the
//   same activation rows, which then stay in that XCD's L2.
// The slot order of the operands and the decode of the weight bytes are the
// format's (formats.h); where the decode leaves a factor 2^kHiLog2 on slots
// 4..7 (Q4_0), the activations of those slots carry 2^-kHiLog2.
#include <algorithm>
#include <atomic>
#include <mutex>
#include <type_traits>

#include "device_common.h"
#include "formats.h"
#include "gemm_split.h"
#include "launch.h"
#include "validate.h"

namespace q4k {

constexpr int kGemmThreads = 256;
constexpr int kEntries = 8 * 4 * 16;   // 16-row subtiles x k-groups x rows: 512 x 16 bytes

struct GemmStage {
    uint4 a[2][kEntries];   // [hi | lo][subtile][g][row] 8-half operands
    uint4 b[2][kEntries];   // [code | code 2^-11][subtile][g][col]
    float d[kGemmBN];
};

// One K segment of the product: a and w point at block kb0 of row 0 (a row
// of a is K floats, a row of w K/32 blocks), and the segment spans nblk
// blocks. row_exp: when not null, row m of the result is scaled back by
// 2^-row_exp[m]; scale_in says whether the kernel scales row m of a by
// 2^row_exp[m] itself (the f32 path) or a was scaled beforehand (the bfloat16
// and Q8_0-activation paths). accumulate: add the segment's result to y.
template <class F>
__global__ __launch_bounds__(kGemmThreads) void k_gemm_any(const float *__restrict__ a,
                                                          const uint8_t *__restrict__ w,
                                                          float *__restrict__ y, int M, int N,
                                                          int K, int nblk, int tiles_m, int tiles_n,
                                                          const int *__restrict__ row_exp,
                                                          int scale_in, int accumulate)
{
    __shared__ GemmStage st[2];

    // Tile order: XCD x (= workgroup id mod 8) takes tiles [x T/8, (x+1) T/8).
    const int T = tiles_m * tiles_n, L = blockIdx.x;
    const int t = (T % 8 == 0) ? (L % 8) * (T / 8) + L / 8 : L;
    const int m0 = (t / tiles_n) * kGemmBM, n0 = (t % tiles_n) * kGemmBN;

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int li = lane & 15, g = lane >> 4;
    const int wm = wave >> 1, wn = wave & 1;
    const size_t row_bytes = (size_t)(K >> 5) * F::kBytes;

    // Staging role: row r of the slab, half h (elements 16h..16h+15 of the
    // activation block; the quant bytes of lane groups 2h and 2h+1 of the
    // weight block).
    const int r = tid >> 1, h = tid & 1;
    const int ar = min(m0 + r, M - 1);
    const float *arow = a + (size_t)ar * K + 16 * h;
    const uint8_t *wrow = w + (size_t)min(n0 + r, N - 1) * row_bytes;
    const int pin = scale_in ? row_exp[ar] : 0;

    float4 av[4];
    uint32_t wx[2][F::kQsDwords];
    uint32_t wdb = 0;
    auto load_step = [&](int kb) {
        const float4 *src = reinterpret_cast<const float4 *>(arow + (size_t)kb * 32);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            av[q] = src[q];
        const uint8_t *bp = wrow + (size_t)kb * F::kBytes;
        load_qs<F>(bp, 2 * h, wx[0]);
        load_qs<F>(bp, 2 * h + 1, wx[1]);
        wdb = load_u16(bp);
    };
    auto store_step = [&](GemmStage &s) {
        const int sub = r >> 4, i = r & 15;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            // Elements 16h + 4q .. + 3 fill one slot half of one lane group.
            // Slots 4..7 meet weights decoded at 2^kHiLog2 x their code: they
            // carry a further 2^-kHiLog2 (exact).
            const int e0 = 16 * h + 4 * q, gg = F::a_group(e0), half = F::a_half(e0);
            const int sh = pin - (half ? F::kHiLog2 : 0);
            const float4 v = av[q];
            const float e[4] = {ldexpf(v.x, sh), ldexpf(v.z, sh), ldexpf(v.y, sh),
                                ldexpf(v.w, sh)};   // slot order 0, 2, 1, 3
            f16x4 hi, lo;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const f16 x = (f16)e[c];
                hi[c] = x;
                lo[c] = (f16)((e[c] - (float)x) * 2048.0f);
            }
            const int idx = (sub * 4 + gg) * 16 + i;
            reinterpret_cast<uint2 *>(&s.a[0][idx])[half] = bitcast<uint2>(hi);
            reinterpret_cast<uint2 *>(&s.a[1][idx])[half] = bitcast<uint2>(lo);
        }
        const f16x8 scale = {(f16)0x1p-11f, (f16)0x1p-11f, (f16)0x1p-11f, (f16)0x1p-11f,
                             (f16)0x1p-11f, (f16)0x1p-11f, (f16)0x1p-11f, (f16)0x1p-11f};
        const f16x8 b0 = F::decode(wx[0], F::kMagic), b1 = F::decode(wx[1], F::kMagic);
        const int idx0 = (sub * 4 + 2 * h) * 16 + i, idx1 = idx0 + 16;
        s.b[0][idx0] = bitcast<uint4>(b0);
        s.b[1][idx0] = bitcast<uint4>(b0 * scale);
        s.b[0][idx1] = bitcast<uint4>(b1);
        s.b[1][idx1] = bitcast<uint4>(b1 * scale);
        if (h == 0)
            s.d[r] = f16_bits_to_f32(wdb);
    };

    f32x4 acc[4][4];
#pragma unroll
    for (int ms = 0; ms < 4; ++ms)
#pragma unroll
        for (int ns = 0; ns < 4; ++ns)
            acc[ms][ns] = (f32x4){0.f, 0.f, 0.f, 0.f};

    load_step(0);
    store_step(st[0]);
    __syncthreads();

    const f32x4 zero4 = {0.f, 0.f, 0.f, 0.f};
    for (int kb = 0; kb < nblk; ++kb) {
        GemmStage &cur = st[kb & 1];
        const bool more = kb + 1 < nblk;
        if (more)
            load_step(kb + 1);

        f16x8 ahi[4], alo[4], bq[4], bs[4];
        float dv[4];
#pragma unroll
        for (int ms = 0; ms < 4; ++ms) {
            const int idx = ((wm * 4 + ms) * 4 + g) * 16 + li;
            ahi[ms] = bitcast<f16x8>(cur.a[0][idx]);
            alo[ms] = bitcast<f16x8>(cur.a[1][idx]);
        }
#pragma unroll
        for (int ns = 0; ns < 4; ++ns) {
            const int idx = ((wn * 4 + ns) * 4 + g) * 16 + li;
            bq[ns] = bitcast<f16x8>(cur.b[0][idx]);
            bs[ns] = bitcast<f16x8>(cur.b[1][idx]);
            dv[ns] = cur.d[(wn * 4 + ns) * 16 + li];
        }
#pragma unroll
        for (int ms = 0; ms < 4; ++ms) {
#pragma unroll
            for (int ns = 0; ns < 4; ++ns) {
                // The small lo products first, the hi products onto them.
                f32x4 c = __builtin_amdgcn_mfma_f32_16x16x32_f16(alo[ms], bs[ns], zero4, 0, 0, 0);
                c = __builtin_amdgcn_mfma_f32_16x16x32_f16(ahi[ms], bq[ns], c, 0, 0, 0);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    acc[ms][ns][q] = fmaf(dv[ns], c[q], acc[ms][ns][q]);
            }
        }
        if (more)
            store_step(st[(kb + 1) & 1]);
        __syncthreads();
    }

    // Lane (li, g) of tile (ms, ns) holds rows 4g..4g+3 of column li.
#pragma unroll
    for (int ms = 0; ms < 4; ++ms) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int m = m0 + wm * 64 + ms * 16 + 4 * g + q;
            if (m >= M)
                continue;
            const int pe = row_exp ? row_exp[m] : 0;
#pragma unroll
            for (int ns = 0; ns < 4; ++ns) {
                const int n = n0 + wn * 64 + ns * 16 + li;
                if (n < N) {
                    float v = ldexpf(acc[ms][ns][q], -pe);
                    if (accumulate)
                        v += y[(size_t)m * N + n];
                    y[(size_t)m * N + n] = v;
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// bfloat16 activations. A bfloat16 value has an 8-bit significand, so once its
// row is scaled by a power of two 2^p that brings the row's largest magnitude
// into [2^15, 2^16), every element within 2^32 of that maximum (2^28 on Q4_0's
// slots 4..7, which carry a further 2^-4) is exactly a binary16 number: one f16
// term per activation replaces the hi / lo pair of the f32 path, and the same
// MFMAs on the same weight decode give products that are exact in f32. The
// result row is scaled back by 2^-p in the epilogue (exact unless it lands in
// the f32 subnormal range). Smaller elements round to the binary16 grid (2^-24
// after scaling, 2^(E - 39) in the row's own units for max |a| in [2^E,
// 2^(E+1))).
//
// * The row's exponent: the largest magnitude is the largest bfloat16 bit
//   pattern with the sign cleared (which orders finite values by magnitude),
//   and p = 15 - E; p = 0 for an all-zero row or one that holds an infinity
//   or NaN.
// * k_row_exp_bf16 (general kernel's shapes): one wavefront per row, all of
//   its loads in flight at once.
// * k_gemm_prep_bf16 (split path): the exponents and the operands in one
//   launch, arranged as k_gemm_prep_f32 (a workgroup per 16-row group and K
//   part, each finding its group's exponents over the whole rows), writing
//   only the hi operand: operand [mt][kb][sub][lane] in the format's slot
//   order, rows past M zero. (One workgroup per 16-row group, without the K
//   parts, was measured slower: at M = 1024 it leaves three quarters of the
//   CUs idle.)
// * k_gemm_prep_bf16_f32 (general kernel's shapes): the scaled activations as
//   f32, row-major (f16(a') is then exact and the lo term 0).

constexpr int kRowExpWaves = 4;

__global__ __launch_bounds__(64 * kRowExpWaves) void k_row_exp_bf16(const uint16_t *__restrict__ a,
                                                                   int *__restrict__ row_exp,
                                                                   int M, int K)
{
    const int lane = threadIdx.x & 63;
    const int m = blockIdx.x * kRowExpWaves + (threadIdx.x >> 6);
    if (m >= M)   // whole wavefronts only
        return;
    const int p = row_exp_from_bits(row_max_bits_bf16(a + (size_t)m * K, K, lane));
    if (lane == 0)
        row_exp[m] = p;
}

// Blocks a wavefront of k_gemm_prep_bf16 takes at a time (the split path has
// an even number of blocks per row): each row's segment is a whole 128-byte
// line.
constexpr int kPrepBlocks = 2;

template <class F>
__device__ __forceinline__ void prep_bf16_pair(const uint16_t *__restrict__ a, int p,
                                               u32x4 *__restrict__ ops, int M, int K, long long R,
                                               int kb0, int lane)
{
    const int nblk = K >> 5;
    const int li = lane & 15, g = lane >> 4;
    const long long m = R * 16 + li;
    f16x8 hi[kPrepBlocks] = {};
    if (m < M) {
        const uint16_t *blk0 = a + m * K + (long long)kb0 * 32;
        uint2 L[kPrepBlocks], H[kPrepBlocks];
#pragma unroll
        for (int u = 0; u < kPrepBlocks; ++u) {
            L[u] = *reinterpret_cast<const uint2 *>(blk0 + u * 32 + F::a_lo(g));
            H[u] = *reinterpret_cast<const uint2 *>(blk0 + u * 32 + F::a_hi(g));
        }
        const int ph = p - F::kHiLog2;   // slots 4..7 carry a further 2^-kHiLog2
#pragma unroll
        for (int u = 0; u < kPrepBlocks; ++u) {
            // Elements 0..3 of a group are the low and high halves of two
            // dwords, in the slot order x, z, y, w of the f32 path.
            const float e[8] = {
                ldexpf(bf16_bits_to_f32(L[u].x & 0xFFFFu), p), ldexpf(bf16_bits_to_f32(L[u].y & 0xFFFFu), p),
                ldexpf(bf16_bits_to_f32(L[u].x >> 16), p),     ldexpf(bf16_bits_to_f32(L[u].y >> 16), p),
                ldexpf(bf16_bits_to_f32(H[u].x & 0xFFFFu), ph), ldexpf(bf16_bits_to_f32(H[u].y & 0xFFFFu), ph),
                ldexpf(bf16_bits_to_f32(H[u].x >> 16), ph),    ldexpf(bf16_bits_to_f32(H[u].y >> 16), ph)};
#pragma unroll
            for (int s = 0; s < 8; ++s)
                hi[u][s] = (f16)e[s];
        }
    }
    u32x4 *dst = ops + ((R >> 3) * nblk + kb0) * slab_ops<true>() + (R & 7) * 64 + lane;
#pragma unroll
    for (int u = 0; u < kPrepBlocks; ++u)
        dst[u * slab_ops<true>()] = bitcast<u32x4>(hi[u]);
}

// The bfloat16 split path's preparation in one launch, arranged as
// k_gemm_prep_f32: workgroup (R, q) finds the 16 rows' exponents of group R
// over the whole rows (one row per wavefront; part 0 writes row_exp), then
// its wavefronts take the pairs of blocks of K part q in turn. Each pair:
// lane (g, li) reads row li's slots of lane group g for both blocks and
// writes their binary16 values (row past M: zeros) in slab order.
template <class F>
__global__ __launch_bounds__(64 * kPrepWaves) void k_gemm_prep_bf16(const uint16_t *__restrict__ a,
                                                                  int *__restrict__ row_exp,
                                                                  u32x4 *__restrict__ ops, int M,
                                                                  int K, int part_blocks)
{
    __shared__ int s_p[16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const long long R = blockIdx.x;
    const int nblk = K >> 5;
    const int kb0 = (int)blockIdx.y * part_blocks, kb1 = min(kb0 + part_blocks, nblk);
    static_assert(kPrepWaves == 16, "one row of the group per wavefront");
    const long long m = R * 16 + wave;
    int pw = 0;
    if (R * 16 < M)
        pw = row_exp_from_bits(row_max_bits_bf16(a + min(m, (long long)M - 1) * K, K, lane));
    if (lane == 0) {
        s_p[wave] = pw;
        if (blockIdx.y == 0 && m < M)
            row_exp[m] = pw;
    }
    __syncthreads();
    const int p = s_p[lane & 15];
    for (int kb = kb0 + kPrepBlocks * wave; kb < kb1; kb += kPrepBlocks * kPrepWaves)
        prep_bf16_pair<F>(a, p, ops, M, K, R, kb, lane);
}

__global__ __launch_bounds__(256) void k_gemm_prep_bf16_f32(const uint16_t *__restrict__ a,
                                                           const int *__restrict__ row_exp,
                                                           float4 *__restrict__ out, int K,
                                                           long long n_quads)
{
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= n_quads)
        return;
    const int p = row_exp[(i * 4) / K];   // K % 32 == 0: a quad never straddles rows
    const uint2 v = reinterpret_cast<const uint2 *>(a)[i];
    out[i] = make_float4(ldexpf(bf16_bits_to_f32(v.x & 0xFFFFu), p),
                         ldexpf(bf16_bits_to_f32(v.x >> 16), p),
                         ldexpf(bf16_bits_to_f32(v.y & 0xFFFFu), p),
                         ldexpf(bf16_bits_to_f32(v.y >> 16), p));
}

// ---------------------------------------------------------------------------
// f32 activations: the row exponents. k_row_exp_f32 (one wavefront per row)
// takes the largest |a| of the row as the largest f32 bit pattern with the
// sign cleared (which orders finite values by magnitude) and sets p = 14 - E
// for a largest magnitude in [2^E, 2^(E+1)); 0 for an all-zero row or one
// that holds an infinity or NaN.

__global__ __launch_bounds__(64 * kRowExpWaves) void k_row_exp_f32(const float *__restrict__ a,
                                                                  int *__restrict__ row_exp,
                                                                  int M, int K)
{
    const int lane = threadIdx.x & 63;
    const int m = blockIdx.x * kRowExpWaves + (threadIdx.x >> 6);
    if (m >= M)   // whole wavefronts only
        return;
    const int p = row_exp_from_bits_f32(row_max_bits_f32(a + (size_t)m * K, K, lane));
    if (lane == 0)
        row_exp[m] = p;
}

// The split path's preparation in one launch: the row exponents and the
// two-term operands (the same values as k_row_exp_f32 and a split per block).
// Workgroup (R, q) takes 16-row group R and K part q (blocks [q L, q L + L)).
// Every element of a row bounds its exponent, so each of a row group's
// workgroups first finds the 16 rows' maxima over the whole row itself (the
// rows stay in L2 after the first reads; repeating the maxima avoids a
// grid-wide dependency), one row per wavefront; part 0 writes them to
// row_exp. Then its sixteen wavefronts split the part's blocks in turn, two
// at a time.

template <class F>
__global__ __launch_bounds__(64 * kPrepWaves) void k_gemm_prep_f32(const float *__restrict__ a,
                                                                 int *__restrict__ row_exp,
                                                                 u32x4 *__restrict__ ahl, int M,
                                                                 int K, int part_blocks)
{
    __shared__ float4 tile[kPrepWaves][16 * 9];
    __shared__ int s_p[16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const long long R = blockIdx.x;
    const int nblk = K >> 5;
    const int kb0 = (int)blockIdx.y * part_blocks, kb1 = min(kb0 + part_blocks, nblk);
    // Row `wave` of the group (a group wholly past M, part of the last tile,
    // needs no exponents: its operands are zeros).
    static_assert(kPrepWaves == 16, "one row of the group per wavefront");
    const long long m = R * 16 + wave;
    int pw = 0;
    if (R * 16 < M)
        pw = row_exp_from_bits_f32(row_max_bits_f32(a + min(m, (long long)M - 1) * K, K, lane));
    if (lane == 0) {
        s_p[wave] = pw;
        if (blockIdx.y == 0 && m < M)
            row_exp[m] = pw;
    }
    __syncthreads();
    const int p = s_p[lane & 15];
    float4 *t = tile[wave];
    int kb = kb0 + wave;
    for (; kb + kPrepWaves < kb1; kb += 2 * kPrepWaves) {
        const SplitRows x0 = split_load(a, M, K, R, kb, lane);
        const SplitRows x1 = split_load(a, M, K, R, kb + kPrepWaves, lane);
        split_store<F>(x0, p, ahl, M, nblk, R, kb, t, lane);
        split_store<F>(x1, p, ahl, M, nblk, R, kb + kPrepWaves, t, lane);
    }
    if (kb < kb1)
        split_store<F>(split_load(a, M, K, R, kb, lane), p, ahl, M, nblk, R, kb, t, lane);
}

template <class F, bool HO>
static hipError_t launch_split_segments(const u32x4 *ops, const uint8_t *w, float *y, int M, int N,
                                        int K, int tiles_m, int tiles_n, const int *row_exp,
                                        hipStream_t s)
{
    const int nblk = K >> 5;
    const KSegments sg = k_segments(nblk, 2);
    const unsigned T = (unsigned)tiles_m * (unsigned)tiles_n;
    for (int i = 0; i < sg.n; ++i) {
        const int kb0 = i * sg.len, nb = min(sg.len, nblk - kb0);
        const hipError_t e = launch_kernel(
            k_gemm_split<F, HO>, dim3(T), dim3(kSplitGemmThreads), 0, s,
            ops + (size_t)kb0 * slab_ops<HO>(), w + (size_t)kb0 * F::kBytes, y, M, N, nblk, nb,
            tiles_m, tiles_n, row_exp, i > 0 ? 1 : 0);
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

template <class F>
static hipError_t launch_any_segments(const float *a, const uint8_t *w, float *y, int M, int N,
                                      int K, int tiles_m, int tiles_n, const int *row_exp,
                                      int scale_in, hipStream_t s)
{
    const int nblk = K >> 5;
    const KSegments sg = k_segments(nblk, 1);
    const unsigned T = (unsigned)tiles_m * (unsigned)tiles_n;
    for (int i = 0; i < sg.n; ++i) {
        const int kb0 = i * sg.len, nb = min(sg.len, nblk - kb0);
        const hipError_t e = launch_kernel(k_gemm_any<F>, dim3(T), dim3(kGemmThreads), 0, s,
                                           a + (size_t)kb0 * 32, w + (size_t)kb0 * F::kBytes, y,
                                           M, N, K, nb, tiles_m, tiles_n, row_exp, scale_in,
                                           i > 0 ? 1 : 0);
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

// workspace: the row exponents (q4v::gemm_row_exp_bytes(M)), then on the split
// path (split: the caller's choice, q4v::gemm_splits_activations(K) with
// M N < 2^31) the two-term operands.
template <class F>
static hipError_t launch_gemm_f(const float *a, const uint8_t *w, float *y, int M, int N, int K,
                                void *workspace, hipStream_t s, bool split)
{
    const int tiles_m = (M + kGemmBM - 1) / kGemmBM, tiles_n = (N + kGemmBN - 1) / kGemmBN;
    const long long T = (long long)tiles_m * tiles_n;
    if (T > 0x7fffffffLL)
        return hipErrorInvalidValue;
    int *row_exp = static_cast<int *>(workspace);
    if (!split) {
        const hipError_t e = launch_kernel(
            k_row_exp_f32, dim3((unsigned)((M + kRowExpWaves - 1) / kRowExpWaves)),
            dim3(64 * kRowExpWaves), 0, s, a, row_exp, M, K);
        if (e != hipSuccess)
            return e;
        return launch_any_segments<F>(a, w, y, M, N, K, tiles_m, tiles_n, row_exp, 1, s);
    }
    u32x4 *ahl = reinterpret_cast<u32x4 *>(static_cast<char *>(workspace) +
                                           q4v::gemm_row_exp_bytes(M));
    // Row groups of every tile (those past M get zero operands).
    const long long groups = (long long)tiles_m * 8;
    const int nblk = K / 32;
    const int part_blocks = prep_part_blocks(groups, nblk, 1);
    const unsigned qn = (unsigned)((nblk + part_blocks - 1) / part_blocks);
    if (groups > 0x7fffffffLL)
        return hipErrorInvalidValue;
    const hipError_t e = launch_kernel(k_gemm_prep_f32<F>, dim3((unsigned)groups, qn),
                                       dim3(64 * kPrepWaves), 0, s, a, row_exp, ahl, M, K,
                                       part_blocks);
    if (e != hipSuccess)
        return e;
    return launch_split_segments<F, false>(ahl, w, y, M, N, K, tiles_m, tiles_n, row_exp, s);
}

template <class F>
static hipError_t launch_gemm_bf16_f(const uint16_t *a, const uint8_t *w, float *y, int M, int N,
                                     int K, void *workspace, hipStream_t s)
{
    const int tiles_m = (M + kGemmBM - 1) / kGemmBM, tiles_n = (N + kGemmBN - 1) / kGemmBN;
    const long long T = (long long)tiles_m * tiles_n;
    if (T > 0x7fffffffLL)
        return hipErrorInvalidValue;
    int *row_exp = static_cast<int *>(workspace);
    void *act = static_cast<char *>(workspace) + q4v::gemm_row_exp_bytes(M);
    hipError_t e;
    if (!q4v::gemm_bf16_splits(M, N, K)) {
        e = launch_kernel(k_row_exp_bf16, dim3((unsigned)((M + kRowExpWaves - 1) / kRowExpWaves)),
                          dim3(64 * kRowExpWaves), 0, s, a, row_exp, M, K);
        if (e != hipSuccess)
            return e;
        const long long n_quads = (long long)M * K / 4;
        const long long grid = (n_quads + 255) / 256;
        if (grid > 0x7fffffffLL)
            return hipErrorInvalidValue;
        e = launch_kernel(k_gemm_prep_bf16_f32, dim3((unsigned)grid), dim3(256), 0, s, a,
                          (const int *)row_exp, static_cast<float4 *>(act), K, n_quads);
        if (e != hipSuccess)
            return e;
        return launch_any_segments<F>((const float *)act, w, y, M, N, K, tiles_m, tiles_n,
                                      row_exp, 0, s);
    }
    // Every 16-row group of the padded tiles (groups past M write zeros), in
    // K parts of whole pairs.
    const long long groups = (long long)tiles_m * 8;
    const int part_blocks = prep_part_blocks(groups, K / 32, kPrepBlocks);
    if (groups > 0x7fffffffLL)
        return hipErrorInvalidValue;
    e = launch_kernel(k_gemm_prep_bf16<F>,
                      dim3((unsigned)groups, (unsigned)((K / 32 + part_blocks - 1) / part_blocks)),
                      dim3(64 * kPrepWaves), 0, s, a, row_exp, static_cast<u32x4 *>(act), M, K,
                      part_blocks);
    if (e != hipSuccess)
        return e;
    return launch_split_segments<F, true>((const u32x4 *)act, w, y, M, N, K, tiles_m, tiles_n,
                                          row_exp, s);
}

// The split kernel stores with 32-bit offsets: M N < 2^31 on its path.
static bool gemm_f32_splits(int M, int N, int K)
{
    return q4v::gemm_splits_activations(K) && (long long)M * N < (1LL << 31);
}

// Rows that one run of launches takes: a grid dimension holds fewer than 2^32
// threads, and the preparations use 64 for a row, or one for four elements
// where bfloat16 or Q8_0 activations are written as f32 (per_quad).
static int gemm_rows_at_once(int M, int K, bool per_quad)
{
    if (M < (1 << 26) - kGemmBM && (!per_quad || (long long)M * K <= (1LL << 34) - 1024))
        return M;
    const long long rows = std::min(1LL << 25, (1LL << 33) / K);
    return (int)(rows >= kGemmBM ? rows / kGemmBM * kGemmBM : rows);   // K < 2^31: at least 4
}

// launch(r0, rows) over the rows of a call, one run after another: each writes
// the workspace that it reads.
template <class Fn>
static hipError_t by_rows(int M, int K, bool per_quad, Fn launch)
{
    const int rows = gemm_rows_at_once(M, K, per_quad);
    hipError_t e = hipSuccess;
    for (long long r0 = 0; r0 < M && e == hipSuccess; r0 += rows)
        e = launch((size_t)r0, (int)std::min((long long)rows, M - r0));
    return e;
}

hipError_t launch_gemm(WeightFormat fmt, const float *a, const uint8_t *w, float *y, int M, int N,
                       int K, void *workspace, hipStream_t s)
{
    const bool split = gemm_f32_splits(M, N, K);
    return by_rows(M, K, false, [&](size_t r0, int rows) {
        const auto f = fmt == WeightFormat::kQ8_0 ? launch_gemm_f<FmtQ8_0> : launch_gemm_f<FmtQ4_0>;
        return f(a + r0 * (size_t)K, w, y + r0 * (size_t)N, rows, N, K, workspace, s, split);
    });
}

// ---------------------------------------------------------------------------
// The f32 GEMM with no workspace argument (q4_gemm, q8_gemm): for callers that
// cannot allocate. Its scratch, the row exponents and two-term operands of one
// chunk of rows, is this file-scope device array, which every GPU the library
// runs on holds (its own copy) until the process ends. On the host the array's
// name denotes a host-side stand-in, not device memory, so host code uses only
// the address hipGetSymbolAddress returns for the device a call runs on,
// looked up once per device (with that device current) and kept.
//
// Rows are taken in chunks whose workspace fits the array: multiples of 128
// rows on the split path, so every 128-row tile computes exactly what it would
// in one launch over all rows (the result equals q4_gemm_ws's bit for bit).
// Every kernel writes the scratch it reads before reading it, so nothing has to
// start at zero; calls that overlap in time on one GPU share the array and
// race.
static __device__ __align__(256) uint8_t scratch[kGemmScratchBytes];

namespace {
constexpr int kScratchDevices = 64;
std::mutex scratch_mu;
std::atomic<void *> scratch_ptr[kScratchDevices];
}  // namespace

// The device address of `scratch` on the device of stream s (the current
// device for the null stream).
static hipError_t scratch_address(hipStream_t s, void **out)
{
    int dev = 0;
    hipError_t e = s ? hipStreamGetDevice(s, &dev) : hipGetDevice(&dev);
    if (e != hipSuccess)
        return e;
    if (dev < 0 || dev >= kScratchDevices)
        return hipErrorInvalidDevice;
    void *p = scratch_ptr[dev].load(std::memory_order_acquire);
    if (!p) {
        std::lock_guard<std::mutex> lock(scratch_mu);
        p = scratch_ptr[dev].load(std::memory_order_relaxed);
        if (!p) {
            int cur = 0;
            if ((e = hipGetDevice(&cur)) != hipSuccess)
                return e;
            if (cur != dev && (e = hipSetDevice(dev)) != hipSuccess)
                return e;
            e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
            if (cur != dev) {
                const hipError_t back = hipSetDevice(cur);
                if (e == hipSuccess)
                    e = back;
            }
            if (e != hipSuccess || !p)
                return e != hipSuccess ? e : hipErrorInvalidSymbol;
            scratch_ptr[dev].store(p, std::memory_order_release);
        }
    }
    *out = p;
    return hipSuccess;
}

hipError_t launch_gemm_noalloc(WeightFormat fmt, const float *a, const uint8_t *w, float *y, int M,
                               int N, int K, hipStream_t s)
{
    void *scr = nullptr;
    hipError_t e = scratch_address(s, &scr);
    if (e != hipSuccess)
        return e;
    bool split = gemm_f32_splits(M, N, K);
    long long rows = 0;
    if (split) {
        // q4v::gemm_workspace_bytes(R, N, K) = pad256(4 R) + R K 4 for R a
        // multiple of 128 (<= 256 + R (K 4 + 4)).
        rows = (long long)((kGemmScratchBytes - 256) / ((size_t)K * 4 + 4)) / kGemmBM * kGemmBM;
        if (rows < kGemmBM)
            split = false;   // K too long for one tile of operands: the general kernel
    }
    if (!split)
        rows = (long long)(kGemmScratchBytes / 4) / 256 * 256;   // the row exponents only
    for (long long r0 = 0; r0 < M; r0 += rows) {
        const int rc = (int)(M - r0 < rows ? M - r0 : rows);
        const float *ac = a + r0 * K;
        float *yc = y + r0 * N;
        e = fmt == WeightFormat::kQ8_0
                ? launch_gemm_f<FmtQ8_0>(ac, w, yc, rc, N, K, scr, s, split)
                : launch_gemm_f<FmtQ4_0>(ac, w, yc, rc, N, K, scr, s, split);
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

hipError_t launch_gemm_bf16(WeightFormat fmt, const uint16_t *a, const uint8_t *w, float *y, int M,
                            int N, int K, void *workspace, hipStream_t s)
{
    return by_rows(M, K, true, [&](size_t r0, int rows) {
        const auto f = fmt == WeightFormat::kQ8_0 ? launch_gemm_bf16_f<FmtQ8_0> : launch_gemm_bf16_f<FmtQ4_0>;
        return f(a + r0 * (size_t)K, w, y + r0 * (size_t)N, rows, N, K, workspace, s);
    });
}

// ---------------------------------------------------------------------------
// Q8_0-quantized activations (a_q: the [M, K/32] Q8_0 block stream, row m's
// blocks contiguous in K order). A dequantized activation q d is an 8-bit code
// times an 11-bit binary16 scale, exact in f32 with at most 18 significant
// bits; the two-term split of the f32 path (hi = f16(v), lo = f16((v - hi)
// 2^11)) holds any such value exactly while it stays inside binary16's range,
// so the f32 GEMM kernels run unchanged on operands made from the blocks.
// * Range: a Q8_0 block can hold up to 128 x 65504 in magnitude. Each row is
//   scaled by the power of two 2^p that puts 128 max_b |d_b| (an upper bound
//   of the row's magnitudes) in [2^14, 2^15), p = 7 - E for the largest |d| in
//   [2^E, 2^(E+1)) (0 for an all-zero row). The scaled values stay below 2^15
//   and the epilogue scales each result row back by 2^-p.
// * row_exp_q8a: one wavefront per row, the largest |d| as the largest
//   binary16 bit pattern with the sign cleared (k_row_exp_q8a off the split
//   path).
// * k_gemm_prep_q8a (split path): the exponents and the split in one launch,
//   arranged as k_gemm_prep_f32; split_q8_block splits as the f32 path
//   (split_store) from the blocks: code q, d 2^p, the product exact in f32,
//   then the same split and operand order.
// * Off the split path: k_q8a_to_f32 writes the scaled values as f32 for
//   k_gemm_any (which takes the same row exponents).

// The exponent of row `row` (nblk Q8_0 blocks), in every lane of the wavefront.
__device__ __forceinline__ int row_exp_q8a(const uint8_t *__restrict__ row, int nblk, int lane)
{
    uint32_t mx = 0;
    for (int b = lane; b < nblk; b += 64)
        mx = max(mx, load_u16(row + (size_t)b * kQ8Bytes) & 0x7FFFu);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        mx = max(mx, (uint32_t)__shfl_xor((int)mx, o));
    int p = 0;
    if (mx != 0 && mx < 0x7C00u) {
        const int ef = (int)(mx >> 10);
        // Subnormal binary16 scales are (mantissa) 2^-24.
        const int E = ef > 0 ? ef - 15 : (31 - __builtin_clz(mx)) - 24;
        p = 7 - E;
    }
    return p;
}

__global__ __launch_bounds__(64 * kRowExpWaves) void k_row_exp_q8a(const uint8_t *__restrict__ aq,
                                                                  int *__restrict__ row_exp, int M,
                                                                  int K)
{
    const int lane = threadIdx.x & 63;
    const int m = blockIdx.x * kRowExpWaves + (threadIdx.x >> 6);
    if (m >= M)   // whole wavefronts only
        return;
    const int nblk = K >> 5;
    const int p = row_exp_q8a(aq + (size_t)m * (size_t)nblk * kQ8Bytes, nblk, lane);
    if (lane == 0)
        row_exp[m] = p;
}

// Signed byte i of a dword as f32.
__device__ __forceinline__ float code_f32(uint32_t x, int i)
{
    return (float)(int8_t)(x >> (8 * i));
}

template <class F>
__device__ __forceinline__ void split_q8_block(const uint8_t *__restrict__ aq, int p,
                                               u32x4 *__restrict__ ahl, int M, int nblk,
                                               long long R, int kb, int lane)
{
    const int li = lane & 15, g = lane >> 4;
    const long long m = R * 16 + li;
    f16x8 hi = {}, lo = {};
    if (m < M) {
        const uint8_t *blk = aq + ((size_t)m * (size_t)nblk + (size_t)kb) * kQ8Bytes;
        const float d = f16_bits_to_f32(load_u16(blk));
        // Slots 4..7 meet weights decoded at 2^kHiLog2 x their code (as in
        // split_store): they carry a further 2^-kHiLog2.
        const float sl = ldexpf(d, p), sh = ldexpf(d, p - F::kHiLog2);
        const uint32_t cl = load_u32_unaligned(blk + 2 + F::a_lo(g));
        const uint32_t ch = load_u32_unaligned(blk + 2 + F::a_hi(g));
        const float e[8] = {code_f32(cl, 0) * sl, code_f32(cl, 2) * sl, code_f32(cl, 1) * sl,
                            code_f32(cl, 3) * sl, code_f32(ch, 0) * sh, code_f32(ch, 2) * sh,
                            code_f32(ch, 1) * sh, code_f32(ch, 3) * sh};
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            const f16 h = (f16)e[s];
            hi[s] = h;
            lo[s] = (f16)((e[s] - (float)h) * 2048.0f);
        }
    }
    const long long mt = R >> 3;
    const long long idx = (mt * nblk + kb) * kOpsPerBlockTile + (R & 7) * 64 + lane;
    ahl[idx] = bitcast<u32x4>(hi);
    ahl[idx + 8 * 64] = bitcast<u32x4>(lo);
}

// The split path's preparation in one launch, arranged as k_gemm_prep_f32:
// workgroup (R, q) finds group R's row exponents from the whole rows' block
// scales (one row per wavefront; part 0 writes row_exp), then its wavefronts
// split the blocks of K part q in turn.
template <class F>
__global__ __launch_bounds__(64 * kPrepWaves) void k_gemm_prep_q8a(const uint8_t *__restrict__ aq,
                                                                 int *__restrict__ row_exp,
                                                                 u32x4 *__restrict__ ahl, int M,
                                                                 int K, int part_blocks)
{
    __shared__ int s_p[16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const long long R = blockIdx.x;
    const int nblk = K >> 5;
    const int kb0 = (int)blockIdx.y * part_blocks, kb1 = min(kb0 + part_blocks, nblk);
    static_assert(kPrepWaves == 16, "one row of the group per wavefront");
    const long long m = R * 16 + wave;
    int pw = 0;
    if (R * 16 < M)
        pw = row_exp_q8a(aq + (size_t)min(m, (long long)M - 1) * (size_t)nblk * kQ8Bytes, nblk, lane);
    if (lane == 0) {
        s_p[wave] = pw;
        if (blockIdx.y == 0 && m < M)
            row_exp[m] = pw;
    }
    __syncthreads();
    const int p = s_p[lane & 15];
    for (int kb = kb0 + wave; kb < kb1; kb += kPrepWaves)
        split_q8_block<F>(aq, p, ahl, M, nblk, R, kb, lane);
}

__global__ __launch_bounds__(256) void k_q8a_to_f32(const uint8_t *__restrict__ aq,
                                                   const int *__restrict__ row_exp,
                                                   float4 *__restrict__ out, int K,
                                                   long long n_quads)
{
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= n_quads)
        return;
    const long long e = i * 4;                    // K % 32 == 0: a quad never straddles blocks
    const long long m = e / K;
    const int k = (int)(e - m * K);
    const uint8_t *blk = aq + ((size_t)m * (size_t)(K >> 5) + (size_t)(k >> 5)) * kQ8Bytes;
    const float s = ldexpf(f16_bits_to_f32(load_u16(blk)), row_exp[m]);
    const uint32_t c = load_u32_unaligned(blk + 2 + (k & 31));
    out[i] = make_float4(code_f32(c, 0) * s, code_f32(c, 1) * s, code_f32(c, 2) * s,
                         code_f32(c, 3) * s);
}

template <class F>
static hipError_t launch_gemm_q8a_f(const uint8_t *aq, const uint8_t *w, float *y, int M, int N,
                                    int K, void *workspace, hipStream_t s)
{
    const int tiles_m = (M + kGemmBM - 1) / kGemmBM, tiles_n = (N + kGemmBN - 1) / kGemmBN;
    const long long T = (long long)tiles_m * tiles_n;
    if (T > 0x7fffffffLL)
        return hipErrorInvalidValue;
    int *row_exp = static_cast<int *>(workspace);
    void *act = static_cast<char *>(workspace) + q4v::gemm_row_exp_bytes(M);
    hipError_t e;
    if (!q4v::gemm_splits_activations(K) || (long long)M * N >= (1LL << 31)) {
        e = launch_kernel(k_row_exp_q8a, dim3((unsigned)((M + kRowExpWaves - 1) / kRowExpWaves)),
                          dim3(64 * kRowExpWaves), 0, s, aq, row_exp, M, K);
        if (e != hipSuccess)
            return e;
        const long long n_quads = (long long)M * K / 4;
        const long long grid = (n_quads + 255) / 256;
        if (grid > 0x7fffffffLL)
            return hipErrorInvalidValue;
        e = launch_kernel(k_q8a_to_f32, dim3((unsigned)grid), dim3(256), 0, s, aq,
                          (const int *)row_exp, static_cast<float4 *>(act), K, n_quads);
        if (e != hipSuccess)
            return e;
        return launch_any_segments<F>((const float *)act, w, y, M, N, K, tiles_m, tiles_n,
                                      row_exp, 0, s);
    }
    const long long groups = (long long)tiles_m * 8;
    const int nblk = K / 32;
    const int part_blocks = prep_part_blocks(groups, nblk, 1);
    if (groups > 0x7fffffffLL)
        return hipErrorInvalidValue;
    e = launch_kernel(k_gemm_prep_q8a<F>,
                      dim3((unsigned)groups, (unsigned)((nblk + part_blocks - 1) / part_blocks)),
                      dim3(64 * kPrepWaves), 0, s, aq, row_exp, static_cast<u32x4 *>(act), M, K,
                      part_blocks);
    if (e != hipSuccess)
        return e;
    return launch_split_segments<F, false>((const u32x4 *)act, w, y, M, N, K, tiles_m, tiles_n,
                                           row_exp, s);
}

hipError_t launch_gemm_q8a(WeightFormat fmt, const uint8_t *a_q, const uint8_t *w, float *y, int M,
                           int N, int K, void *workspace, hipStream_t s)
{
    return by_rows(M, K, true, [&](size_t r0, int rows) {
        const auto f = fmt == WeightFormat::kQ8_0 ? launch_gemm_q8a_f<FmtQ8_0> : launch_gemm_q8a_f<FmtQ4_0>;
        return f(a_q + r0 * ((size_t)(K / 32) * kQ8Bytes), w, y + r0 * (size_t)N, rows, N, K, workspace, s);
    });
}

}  // namespace q4k
