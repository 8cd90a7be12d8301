// Products grouped by expert over Q4_0 and Q8_0 weights, f32 or bfloat16
// activations: y[r] = a[r / share] @ dequant(W[e])^T for the rows r of each
// group e (groups.h), each group with its own number of rows.
//
// The arithmetic is the GEMM's (gemm.hip): a row of activations is scaled by
// a power of two and written once as binary16 matrix-core operands (two terms
// of f32, one of bfloat16), weights decode to exact binary16 codes, and every
// block's sum is scaled by its d in f32. What is new is where rows and weights
// come from, and a form for few rows.
//
// The preparation gathers the rows: each group's rows fill tiles of bm rows,
// the last one short; operands [tile][block][term][16-row subtile][lane], row
// exponents [tile row].
#include "device_common.h"
#include "formats.h"
#include "gemm_split.h"
#include "gemv_stream.h"
#include "groups.h"
#include "launch.h"
#include "validate.h"

namespace q4k {

// Workgroup (x, q): 16-row subtile x of the tiles, K part q. One wavefront per
// row finds the row's exponent over the whole row, then the wavefronts take
// the part's blocks in turn, lane (g, li) the slots of lane group g of row li.
// Subtiles past a group's last row write nothing: their operands reach only
// rows of y that are not stored.
template <class F, bool BF, int BM>
__global__ __launch_bounds__(64 * kPrepWaves) void k_grouped_prep(const void *__restrict__ a,
                                                                Groups gr, int *__restrict__ row_exp,
                                                                u32x4 *__restrict__ ops, int K,
                                                                int part_blocks, int *__restrict__ claims,
                                                                int N, int first)
{
    __shared__ int s_p[16], s_row[16];
    __shared__ u32x4 s_tile[kPrepWaves][16 * 9];
    constexpr int SUBS = BM / 16, TERMS = BF ? 1 : 2;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int x = first + (int)blockIdx.x, t = x / SUBS, sub = x % SUBS;
    const GroupTile gt = find_group_tile(gr, t, BM, 1);
    const int p0 = gt.lo + gt.mt * BM + sub * 16;
    if (gt.e < 0 || p0 >= gt.hi)
        return;
    const float *af = static_cast<const float *>(a);
    const uint16_t *ab = static_cast<const uint16_t *>(a);
    const int r = p0 + wave < gt.hi ? group_row(gr, p0 + wave) : -1;
    int p = 0;
    if (r >= 0) {
        const size_t at = (size_t)(r / gr.share) * (size_t)K;
        p = BF ? row_exp_from_bits(row_max_bits_bf16(ab + at, K, lane))
               : row_exp_from_bits_f32(row_max_bits_f32(af + at, K, lane));
    }
    if (lane == 0) {
        s_p[wave] = p;
        s_row[wave] = r;
        if (blockIdx.y == 0) {
            row_exp[(size_t)t * BM + sub * 16 + wave] = p;
            if (claims && r >= 0)
                claims[(size_t)r * (size_t)N] = t * BM + sub * 16 + wave;
        }
    }
    __syncthreads();
    // A unit is 128 bytes of each row. Eight lanes read a row's, whole lines,
    // and a padded LDS tile hands lane (g, li) its slots (4096 rows of 4096
    // bfloat16: 26.4 us when each lane reads its own slots, 18.5 so; 512 of f32
    // 13.4 and 9.2).
    constexpr int ES = BF ? 2 : 4, UB = BF ? 2 : 1;
    const int nblk = K >> 5;
    const int kb0 = (int)blockIdx.y * part_blocks, kb1 = min(kb0 + part_blocks, nblk);
    const int pr = lane >> 3, pc = lane & 7;
    const char *src[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        src[i] = static_cast<const char *>(a) + (size_t)(max(s_row[pr + 8 * i], 0) / gr.share) * (size_t)K * ES + pc * 16;
    const int li = lane & 15, g = lane >> 4;
    const int pl = s_p[li], ph = pl - F::kHiLog2;
    const bool there = s_row[li] >= 0;
    u32x4 *tile = s_tile[wave];
    int kb = kb0 + UB * wave;
    u32x4 v[2];
    auto load = [&](int b) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            v[i] = *reinterpret_cast<const u32x4 *>(src[i] + (size_t)b * (32 * ES));
    };
    if (kb < kb1)
        load(kb);
    for (; kb < kb1; kb += UB * kPrepWaves) {
        wave_lds_fence();   // the previous unit has been read
#pragma unroll
        for (int i = 0; i < 2; ++i)
            tile[(pr + 8 * i) * 9 + pc] = v[i];
        wave_lds_fence();
        if (kb + UB * kPrepWaves < kb1)
            load(kb + UB * kPrepWaves);
#pragma unroll
        for (int u = 0; u < UB; ++u) {
            float e[8];
            if constexpr (BF) {
                const uint2 *t = reinterpret_cast<const uint2 *>(tile + li * 9) + u * 8;
                const uint2 L = t[F::a_lo(g) / 4], H = t[F::a_hi(g) / 4];
                const float x[8] = {bf16_bits_to_f32(L.x & 0xFFFFu), bf16_bits_to_f32(L.y & 0xFFFFu),
                                    bf16_bits_to_f32(L.x >> 16), bf16_bits_to_f32(L.y >> 16),
                                    bf16_bits_to_f32(H.x & 0xFFFFu), bf16_bits_to_f32(H.y & 0xFFFFu),
                                    bf16_bits_to_f32(H.x >> 16), bf16_bits_to_f32(H.y >> 16)};
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    e[s] = ldexpf(x[s], s < 4 ? pl : ph);
            } else {
                const float4 L = *reinterpret_cast<const float4 *>(tile + li * 9 + F::a_lo(g) / 4);
                const float4 H = *reinterpret_cast<const float4 *>(tile + li * 9 + F::a_hi(g) / 4);
                const float x[8] = {L.x, L.z, L.y, L.w, H.x, H.z, H.y, H.w};
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    e[s] = ldexpf(x[s], s < 4 ? pl : ph);
            }
            f16x8 hi, lo;
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const float x = there ? e[s] : 0.0f;
                const f16 h = (f16)x;
                hi[s] = h;
                lo[s] = (f16)((x - (float)h) * 2048.0f);
            }
            u32x4 *dst = ops + (((size_t)t * nblk + kb + u) * TERMS * SUBS + sub) * 64 + lane;
            dst[0] = bitcast<u32x4>(hi);
            if constexpr (!BF)
                dst[SUBS * 64] = bitcast<u32x4>(lo);
        }
    }
}

// Where K is cut into segments, every launch after the first adds to y, so a row
// that the lists name more than once must be one tile row's alone. Each tile
// row leaves its number in its row of y in the preparation (the first element,
// until the product stores there), and those whose number is not the one that
// stayed are marked in row_exp: 4.6 us beside products of some hundred. Which
// one stays is left open. Workgroup t: tile t.
__global__ __launch_bounds__(kGemmBM) void k_grouped_resolve(Groups gr, const int *__restrict__ claims, int N,
                                                            int *__restrict__ row_exp)
{
    const GroupTile gt = find_group_tile(gr, blockIdx.x, kGemmBM, 1);
    const int p = gt.lo + gt.mt * kGemmBM + (int)threadIdx.x, j = (int)(blockIdx.x * kGemmBM + threadIdx.x);
    const int r = gt.e >= 0 && p < gt.hi ? group_row(gr, p) : -1;
    if (r >= 0 && claims[(size_t)r * (size_t)N] != j)
        row_exp[j] = kNotStored;
}

template <class F, bool HO>
__global__ __launch_bounds__(kSplitGemmThreads) void k_gemm_split_grouped(
    const u32x4 *__restrict__ ahl, const uint8_t *__restrict__ w, float *__restrict__ y, int N,
    int nblk_row, int nblk, int tiles_n, const int *__restrict__ row_exp, int accumulate, Groups gr,
    int first)
{
    __shared__ SplitLds<F, HO> lds;
    const GroupTile gt = find_group_tile(gr, xcd_runs(first + (int)blockIdx.x), kGemmBM, tiles_n);
    if (gt.e < 0 || gt.before + gt.mt >= gr.tiles)
        return;
    if constexpr (HO) {
        // A group's last tile computes a half or a quarter of its rows where it
        // has no more.
        const int rows = gt.hi - gt.lo - gt.mt * kGemmBM;
        if (rows <= 32) {
            gemm_split_body<F, HO, true, 2>(ahl, w, y, 0, N, nblk_row, nblk, 0, tiles_n, row_exp, accumulate, gr, gt, lds);
            return;
        }
        if (rows <= 64) {
            gemm_split_body<F, HO, true, 4>(ahl, w, y, 0, N, nblk_row, nblk, 0, tiles_n, row_exp, accumulate, gr, gt, lds);
            return;
        }
    }
    gemm_split_body<F, HO, true>(ahl, w, y, 0, N, nblk_row, nblk, 0, tiles_n, row_exp, accumulate, gr, gt, lds);
}

// ---------------------------------------------------------------------------
// Few rows a group: bound by the bytes of the weights. Workgroup (x, t) takes
// 16 CT weight rows past one pass, up to 16 R rows of a group: a long group's
// passes run side by side and share its weights in L2 (487 tokens, 2 of 32
// experts unevenly, 1882 x 320: 37 us with one workgroup for all of a group's
// passes, 27 so). Its four wavefronts deal the row's chunks of 8 blocks (256
// elements: 144 or 272 bytes, whole 16-byte pieces; the last one may be short)
// among themselves; each stages its own chunk's raw bytes in its own LDS by
// 16-byte direct loads (rows need dword alignment only: K % 64 == 0), one chunk
// ahead, and so waits only for its own loads, never for the others. A row of a
// staged chunk is 36 or 68 dwords, 4 mod 32, so the sixteen rows an operand read
// touches lie in different banks. The activation operands of a chunk go from L2 to
// registers (they are the wavefront's own: no other reads that chunk), once
// for all 16 CT weight rows. The partial tiles are added through LDS. Four
// wavefronts, so that two workgroups share a compute unit and one streams while
// the other decodes or adds up (37 tokens, 2 of 8 experts, 14336 x 4096: Q8_0
// 154 -> 128 us, Q4_0 with f32 activations 118 -> 106, 100 tokens of bfloat16
// 134 -> 124). Also measured, and no faster (90-100 us of Q4_0, bfloat16):
// persistent workgroups with the loads running on into the next tile, three
// stages, loads spread between the blocks' decodes. Of its 73 us the bytes
// need 56 and the decode's issue (14 vector instructions a matrix instruction,
// 917504 of these) some 22: what is left is latency, with two wavefronts a SIMD
// (74 KB of LDS a workgroup) to hide it.
constexpr int kFewWaves = 4, kFewBlocks = 8;

template <class F, int CT>
struct FewGeom {
    static constexpr int kRowBytes = kFewBlocks * F::kBytes;    // of a chunk
    static constexpr int kPieces = kRowBytes / 16;
    static constexpr int kRows = 16 * CT;
    static constexpr int kLoads = (kRows * kPieces + 63) / 64;  // 16-byte loads of a wavefront per chunk
    static constexpr int kStage = kLoads * 64;                  // 16-byte LDS words
};

template <class F, bool HO, int CT, int R>
struct FewLds {
    union {
        u32x4 w[kFewWaves][2][FewGeom<F, CT>::kStage];
        f32x4 red[kFewWaves][R * CT][64];
    };
    int row[64], exp[64];   // of the 16 R rows
};

// Pass t over the groups one after another, 16 R rows a pass (the last of a
// group shorter): its group, its positions from lo on (hi: the group's end) and
// its first 16-row tile. At most 2^15 tiles a group here: the sums stay small
// whatever the lists hold.
struct FewPass {
    int e, lo, hi, tile;
};

__device__ __forceinline__ FewPass find_pass(const Groups &gr, int t, int R)
{
    const int lane = threadIdx.x & 63;
    int passes = 0, tiles = 0;   // of the groups before base
    for (int base = 0; base < gr.G; base += 64) {
        int lo = 0, hi = 0;
        if (base + lane < gr.G)
            group_bounds(gr, base + lane, lo, hi);
        const int mine = (hi - lo + 15) / 16, my_passes = (mine + R - 1) / R;
        int st = mine, sp = my_passes;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int vt = __shfl_up(st, d), vp = __shfl_up(sp, d);
            if (lane >= d)
                st += vt, sp += vp;
        }
        const uint64_t past = __ballot(passes + sp > t);
        if (past) {
            const int l = __builtin_ctzll(past);
            const int k = t - passes - __builtin_amdgcn_readlane(sp - my_passes, l);
            return {base + l, __builtin_amdgcn_readlane(lo, l) + k * 16 * R, __builtin_amdgcn_readlane(hi, l),
                    tiles + __builtin_amdgcn_readlane(st - mine, l) + k * R};
        }
        passes += __builtin_amdgcn_readlane(sp, 63);
        tiles += __builtin_amdgcn_readlane(st, 63);
    }
    return {-1, 0, 0, 0};
}

template <class F, bool HO, int CT, int R>
__global__ __launch_bounds__(64 * kFewWaves) void k_grouped_few(const u32x4 *__restrict__ ops,
                                                              const int *__restrict__ row_exp,
                                                              const uint8_t *__restrict__ w,
                                                              float *__restrict__ y, int N, int K,
                                                              Groups gr, int first)
{
    using G = FewGeom<F, CT>;
    constexpr int TERMS = HO ? 1 : 2;
    __shared__ FewLds<F, HO, CT, R> lds;
    const FewPass at = find_pass(gr, blockIdx.y, R);
    if (at.e < 0 || at.tile >= gr.tiles)
        return;
    const int e = at.e, lo = at.lo, hi = at.hi, tile = at.tile;
    const int subs = min(min(R, (hi - lo + 15) / 16), gr.tiles - tile);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int li = lane & 15, g = lane >> 4;
    const int nblk = K >> 5, chunks = (nblk + kFewBlocks - 1) / kFewBlocks;
    const int n0 = (first + (int)blockIdx.x) * G::kRows;
    const uint32_t row_bytes = (uint32_t)nblk * F::kBytes;
    const int wrows = min(G::kRows, N - n0);
    // At most 64 rows of 14336 elements: the offsets are far below 2^31.
    const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(w + ((size_t)e * (size_t)N + (size_t)n0) * (size_t)row_bytes), (short)0,
        (int)((uint32_t)wrows * row_bytes), kBufferRsrcWord3);
    uint32_t off[G::kLoads];
#pragma unroll
    for (int j = 0; j < G::kLoads; ++j) {
        const int t = min(j * 64 + lane, G::kRows * G::kPieces - 1);   // surplus lanes re-read the last piece
        const int row = t / G::kPieces;
        off[j] = (uint32_t)min(row, wrows - 1) * row_bytes + 16u * (uint32_t)(t - row * G::kPieces);
    }
    // At most 2^19 rows here, and gr.tiles tiles of 16 exponents.
    const __amdgpu_buffer_rsrc_t orders = __builtin_amdgcn_make_buffer_rsrc(
        (void *)gr.order, (short)0, gr.order ? gr.M * 4 : 0, kBufferRsrcWord3);
    const __amdgpu_buffer_rsrc_t exps = __builtin_amdgcn_make_buffer_rsrc(
        (void *)row_exp, (short)0, gr.tiles * 64, kBufferRsrcWord3);
    const uint32_t magic = magic_vgpr<F>();
    auto issue = [&](int c, int buf) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < G::kLoads; ++j)
            load16_to_lds(wr, lds.w[wave][buf] + j * 64, off[j], c * G::kRowBytes);
    };
    const f16 sc = (f16)0x1p-11f;
    const f16x8 scale = {sc, sc, sc, sc, sc, sc, sc, sc};
    const f32x4 zero4 = {0.f, 0.f, 0.f, 0.f};

    f32x4 acc[R][CT];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
            acc[r][ct] = zero4;
    // The rows of y and their exponents arrive while the weights stream (37
    // tokens, 2 of 8 experts, 14336 x 4096, Q4_0: 96 us when they are read one
    // by one behind the last chunk, 93 so).
    if (wave == 0) {
        const uint32_t i = (uint32_t)lane * 4u;
        if (gr.order)
            load4_to_lds(orders, lds.row, i, lo * 4);
        load4_to_lds(exps, lds.exp, lane < 16 * subs ? i : 0u, tile * 64);
    }
    const int last = chunks - 1;
    if (wave < chunks) {
        issue(wave, 0);
        int buf = 0;
        // This chunk's operands, then the next chunk's bytes: waiting for
        // the operands leaves those in flight. Past the last chunk the
        // last one is read again, into the buffer nobody reads.
        auto chunk = [&](auto full_c, int c) __attribute__((always_inline)) {
            constexpr bool full = decltype(full_c)::value;
            const int left = nblk - c * kFewBlocks;   // blocks of a short last chunk
            f16x8 aop[R][TERMS][kFewBlocks];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const u32x4 *src = ops + ((size_t)(tile + min(r, subs - 1)) * nblk + c * kFewBlocks) * (TERMS * 64) + lane;
#pragma unroll
                for (int b = 0; b < kFewBlocks; ++b)
#pragma unroll
                    for (int h = 0; h < TERMS; ++h)
                        aop[r][h][b] = bitcast<f16x8>(src[((full ? b : min(b, left - 1)) * TERMS + h) * 64]);
            }
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(63));   // the other buffer has been read
            issue(min(c + kFewWaves, last), buf ^ 1);
            __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(G::kLoads));
            asm volatile("" ::: "memory");
            const uint32_t *base = reinterpret_cast<const uint32_t *>(lds.w[wave][buf]) + li * (G::kRowBytes / 4);
            unroll<kFewBlocks>([&](auto b_c) __attribute__((always_inline)) {
                constexpr int b = decltype(b_c)::value;
                if (!full && b >= left)
                    return;
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    const uint32_t *row = base + ct * 16 * (G::kRowBytes / 4);
                    uint32_t x[F::kQsDwords];
                    read_qs<F, b>(row, g, x);
                    const float d = f16_bits_to_f32(read_d_bits<F, b>(row));
                    const f16x8 q = F::decode(x, magic);
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        f32x4 s = zero4;
                        if constexpr (!HO)
                            s = __builtin_amdgcn_mfma_f32_16x16x32_f16(aop[r][1][b], q * scale, s, 0, 0, 0);
                        s = __builtin_amdgcn_mfma_f32_16x16x32_f16(aop[r][0][b], q, s, 0, 0, 0);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc[r][ct][i] = fmaf(d, s[i], acc[r][ct][i]);
                    }
                }
            });
            buf ^= 1;
        };
        for (int c = wave; c < chunks; c += kFewWaves) {
            if (c < chunks - 1 || nblk % kFewBlocks == 0)
                chunk(std::true_type{}, c);
            else
                chunk(std::false_type{}, c);
        }
    }
    // Every load has landed before its LDS serves the partial tiles.
    ring_barrier<0>();
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
            lds.red[wave][r * CT + ct][lane] = acc[r][ct];
    __syncthreads();
    for (int i = wave; i < R * CT; i += kFewWaves) {
        const int r = i / CT, ct = i % CT, n = n0 + ct * 16 + li;
        f32x4 v = lds.red[0][i][lane];
#pragma unroll
        for (int s = 1; s < kFewWaves; ++s)
            v += lds.red[s][i][lane];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int j = 16 * r + 4 * g + q, row = gr.order ? lds.row[j] : lo + j;
            if (r < subs && lo + j < hi && (unsigned)row < (unsigned)gr.M && n < N)
                y[(size_t)row * (size_t)N + n] = ldexpf(v[q], -lds.exp[j]);
        }
    }
}

// One to eight rows in all (grouped_in_place): each is a decode GEMV of one
// activation row (gemv_stream.h) with its group's weights, in one launch, with
// no preparation and no workspace. Workgroup (x, p) takes 16 weight rows for
// position p; rows of one group read its weights once each, which costs more
// only where such rows are many.
template <class F, bool BF, int CH, bool LA>
__global__ __launch_bounds__(64 * kGemvStreamWaves) void k_grouped_gemv(const void *__restrict__ a,
                                                                      const uint8_t *__restrict__ w,
                                                                      float *__restrict__ y, int N,
                                                                      int K, Groups gr)
{
    const int p = blockIdx.y;
    int e = -1;
    for (int base = 0; base < gr.G && e < 0; base += 64) {
        int lo = 0, hi = 0;
        if (base + (int)(threadIdx.x & 63) < gr.G)
            group_bounds(gr, base + (int)(threadIdx.x & 63), lo, hi);
        const uint64_t in = __ballot(lo <= p && p < hi);
        if (in)
            e = base + __builtin_ctzll(in);
    }
    const int row = __builtin_amdgcn_readfirstlane(group_row(gr, p));
    if (e < 0 || row < 0)
        return;
    const int nblk = K >> 5;
    gemv_stream_body<F, 1, kGemvStreamWaves, CH, BF, 1, 16, LA, false, LA>(
        static_cast<const uint8_t *>(a) + (size_t)(row / gr.share) * (size_t)K * (BF ? 2 : 4),
        w + (size_t)e * (size_t)N * ((size_t)nblk * F::kBytes), y + (size_t)row * (size_t)N, N, K,
        nblk, 0);
}

template <class F, bool BF, bool LA>
static hipError_t launch_grouped_gemv(const void *a, const uint8_t *w, float *y, int N, int K,
                                      const Groups &gr, hipStream_t s)
{
    return launch_kernel(q4v::gemv_chunk_blocks(K / 32, K / 32) == 16 ? k_grouped_gemv<F, BF, 16, LA>
                                                                     : k_grouped_gemv<F, BF, 8, LA>,
                         dim3((unsigned)((N + 15LL) / 16), (unsigned)gr.M), dim3(64 * kGemvStreamWaves),
                         0, s, a, w, y, N, K, gr);
}

template <class F, bool BF, int CT, int R>
static hipError_t launch_few(const u32x4 *ops, const int *row_exp, const uint8_t *w, float *y,
                             int N, int K, const Groups &gr, hipStream_t s)
{
    static_assert(sizeof(FewLds<F, BF, CT, R>) <= (size_t)kLdsBytes, "the stages fit in LDS");
    return launch_parts(k_grouped_few<F, BF, CT, R>, (N + 16LL * CT - 1) / (16 * CT),
                        (unsigned)q4v::group_row_tiles(gr.G, gr.M, 16 * R), 64 * kFewWaves, s, ops, row_exp, w, y,
                        N, K, gr);
}

template <class F, bool BF>
static hipError_t launch_grouped_f(const void *a, const uint8_t *w, float *y, int N, int K,
                                   const Groups &gr, void *workspace, hipStream_t s)
{
    if (q4v::grouped_in_place(gr.M, N, K, F::kBytes, BF ? 2 : 4))
        return gemv_rows_line_aligned<F>(w, K) ? launch_grouped_gemv<F, BF, true>(a, w, y, N, K, gr, s)
                                               : launch_grouped_gemv<F, BF, false>(a, w, y, N, K, gr, s);
    const bool few = q4v::grouped_few(gr.G, gr.M, N, K);
    const int bm = few ? 16 : 128, nblk = K >> 5;
    const long long tiles = q4v::group_row_tiles(gr.G, gr.M, bm);
    int *row_exp = static_cast<int *>(workspace);
    u32x4 *ops = reinterpret_cast<u32x4 *>(static_cast<char *>(workspace) + q4v::grouped_exp_bytes(gr.G, gr.M, N, K));
    const long long groups = tiles * (bm / 16);
    const int part = prep_part_blocks(groups, nblk, BF ? 2 : 1);
    const KSegments sg = few ? KSegments{1, nblk} : k_segments(nblk, 2);
    int *claims = sg.n > 1 ? reinterpret_cast<int *>(y) : nullptr;
    hipError_t e = launch_parts(few ? k_grouped_prep<F, BF, 16> : k_grouped_prep<F, BF, 128>, groups,
                                (unsigned)((nblk + part - 1) / part), 64 * kPrepWaves, s, a, gr, row_exp,
                                ops, K, part, claims, N);
    if (e != hipSuccess)
        return e;
    if (few) {
        constexpr int CTL = F::kBytes == kQ8Bytes ? 2 : 4;
        const q4v::FewShape fs = q4v::grouped_few_shape(gr.G, gr.M, N, F::kBytes);
        if (fs.ct == CTL)
            return fs.r == 2 ? launch_few<F, BF, CTL, 2>(ops, row_exp, w, y, N, K, gr, s)
                             : launch_few<F, BF, CTL, 1>(ops, row_exp, w, y, N, K, gr, s);
        return launch_few<F, BF, 1, 1>(ops, row_exp, w, y, N, K, gr, s);
    }
    const long long tn = ((long long)N + kGemmBN - 1) / kGemmBN;
    const long long grid = group_grid(gr.G, gr.M, kGemmBM, tn);
    if (grid > kMaxGroupTiles)
        return hipErrorInvalidValue;
    if (claims) {
        e = launch_kernel(k_grouped_resolve, dim3((unsigned)tiles), dim3(kGemmBM), 0, s, gr,
                          (const int *)claims, N, row_exp);
        if (e != hipSuccess)
            return e;
    }
    for (int i = 0; i < sg.n; ++i) {
        const int kb0 = i * sg.len, nb = min(sg.len, nblk - kb0);
        e = launch_parts(k_gemm_split_grouped<F, BF>, grid, 1, kSplitGemmThreads, s,
                         (const u32x4 *)(ops + (size_t)kb0 * slab_ops<BF>()),
                         w + (size_t)kb0 * F::kBytes, y, N, nblk, nb, (int)tn,
                         (const int *)row_exp, i > 0 ? 1 : 0, gr);
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

hipError_t launch_gemm_grouped(WeightFormat fmt, bool bf16, const void *a, const uint8_t *w,
                               const int *offsets, const int *order, int share, float *y, int G,
                               int M, int N, int K, void *workspace, hipStream_t s)
{
    const int bm = q4v::grouped_few(G, M, N, K) ? 16 : 128;
    const Groups gr = {offsets, order, G, M, share, (int)q4v::group_row_tiles(G, M, bm)};
    if (fmt == WeightFormat::kQ8_0)
        return bf16 ? launch_grouped_f<FmtQ8_0, true>(a, w, y, N, K, gr, workspace, s)
                    : launch_grouped_f<FmtQ8_0, false>(a, w, y, N, K, gr, workspace, s);
    return bf16 ? launch_grouped_f<FmtQ4_0, true>(a, w, y, N, K, gr, workspace, s)
                : launch_grouped_f<FmtQ4_0, false>(a, w, y, N, K, gr, workspace, s);
}

}  // namespace q4k
