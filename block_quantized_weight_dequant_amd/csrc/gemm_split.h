// The GEMM's split-activation kernel and what its preparation shares, for the
// plain GEMM (gemm.hip) and the products grouped by expert (grouped.hip).
#pragma once

#include <climits>
#include <type_traits>

#include "device_common.h"
#include "formats.h"
#include "groups.h"

namespace q4k {

constexpr int kGemmBM = 128;
constexpr int kGemmBN = 128;

// ---------------------------------------------------------------------------
// Split-activation path, for K % 64 == 0 (K splits into pairs of blocks, and a
// weight row, a whole number of pairs of 36 or 68 bytes, starts on a 4-byte
// boundary).
//
// * k_gemm_prep_f32 finds the row exponents and writes the activations once,
//   already split (hi = f16(a), lo = f16((a - hi) 2^11), after the row's power
//   of two) and laid out as the matrix cores' A operands:
//   16-byte operand [mt][kb][hl][sub][lane] holds, for row 128 mt + 16 sub +
//   lane % 16 and block kb, the slots of lane group g = lane / 16 in the
//   format's order (formats.h), hi for hl = 0 and lo for hl = 1. Rows past M
//   are zero. The split then costs one pass over the activations instead of
//   one per column tile, and a workgroup's activation slab for a pair of
//   blocks is 32 contiguous KB.
// * k_gemm_split: a 512-thread workgroup computes a 128 x 128 tile. Its eight
//   wavefronts are two K groups of four: group kg takes the even (kg = 0) or
//   odd (kg = 1) block of each pair, and wavefront (wm, wn) of a group owns a
//   64 x 64 quadrant as 4 x 4 MFMA tiles. Two wavefronts per SIMD hide each
//   other's VALU work and latencies; the two groups' partial tiles are added
//   once, through LDS, at the end.
// * Per pair of blocks the workgroup stages the 32 KB activation slab and the
//   raw weight bytes of the pair (36 or 68 per row) of its 128 rows in LDS,
//   with direct-to-LDS loads in a ring (below). Each wavefront decodes its own
//   B operands from the raw bytes: the quant bytes of lane group g for column
//   lane % 16, realigned with v_alignbyte where they straddle dwords, become
//   the binary16 codes and the same times 2^-11, and d stays binary16 until
//   the scale FMA.
// * Accumulation as in the general kernel: two chained MFMAs per 16 x 16 tile
//   and block (lo x code 2^-11, then hi x code onto it), then d * C + acc in
//   f32.

constexpr int kOpsPerBlockTile = 2 * 8 * 64;   // 16-byte A operands per (128-row tile, block)

// The one-launch preparations (k_gemm_prep_f32, k_gemm_prep_bf16,
// k_gemm_prep_q8a): one wavefront per row of a 16-row group.
constexpr int kPrepWaves = 16;
constexpr long long kPrepTarget = 256;   // workgroups the preparation aims for

// Blocks per K part of a fused preparation: enough parts for about
// kPrepTarget workgroups over `groups` row groups, each part a whole number
// of `unit` blocks and at least one unit per wavefront.
inline int prep_part_blocks(long long groups, int nblk, int unit)
{
    const long long units = nblk / unit;
    const long long parts = max(1LL, min(units / kPrepWaves, (kPrepTarget + groups - 1) / groups));
    return (int)((units + parts - 1) / parts) * unit;
}

// Order a wavefront's LDS writes before its later LDS reads (its LDS
// operations execute in issue order; the fences keep the compiler's order).
__device__ __forceinline__ void wave_lds_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The split of one (16-row group R, block kb) by one wavefront: lane l loads
// 16-byte piece l % 8 of rows l / 8 and 8 + l / 8 (whole 128-byte block rows,
// eight lanes per row; rows past M re-read row M - 1 and are written as
// zeros), and a padded LDS tile ([16 rows][9 pieces]: conflict-free both
// ways) hands lane (g, li) its two pieces, the slots of lane group g of row
// li, which it splits with row li's power of two p.
struct SplitRows {
    float4 v[2];
};

__device__ __forceinline__ SplitRows split_load(const float *__restrict__ a, int M, int K,
                                                long long R, int kb, int lane)
{
    const int pr = lane >> 3, pc = lane & 7;
    SplitRows x;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const long long row = min(R * 16 + pr + 8 * i, (long long)M - 1);
        x.v[i] = *reinterpret_cast<const float4 *>(a + row * K + (long long)kb * 32 + 4 * pc);
    }
    return x;
}

template <class F>
__device__ __forceinline__ void split_store(const SplitRows &x, int p, u32x4 *__restrict__ ahl,
                                            int M, int nblk, long long R, int kb, float4 *tile,
                                            int lane)
{
    const int pr = lane >> 3, pc = lane & 7;
    wave_lds_fence();   // the tile's previous reads precede these writes
#pragma unroll
    for (int i = 0; i < 2; ++i)
        tile[(pr + 8 * i) * 9 + pc] = x.v[i];
    wave_lds_fence();
    const int li = lane & 15, g = lane >> 4;
    const long long m = R * 16 + li;
    f16x8 hi = {}, lo = {};
    if (m < M) {
        const float4 L = tile[li * 9 + F::a_lo(g) / 4];
        const float4 H = tile[li * 9 + F::a_hi(g) / 4];
        // Slots 4..7 meet weights decoded at 2^kHiLog2 x their code: they carry
        // a further 2^-kHiLog2 (exact), so every product is a 2^p times the code.
        const int ph = p - F::kHiLog2;
        const float e[8] = {ldexpf(L.x, p),  ldexpf(L.z, p),  ldexpf(L.y, p),  ldexpf(L.w, p),
                            ldexpf(H.x, ph), ldexpf(H.z, ph), ldexpf(H.y, ph), ldexpf(H.w, ph)};
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

constexpr int kSplitGemmThreads = 512;
// Word 3 of a raw (untyped, stride 0) buffer resource on gfx9: 32-bit data format.
constexpr int kBufferRsrcWord3 = 0x00020000;
constexpr int kLdsBytes = 160 * 1024;   // LDS of one gfx950 compute unit

// Per-format geometry of one pair of blocks.
template <class F>
struct PairGeom {
    static constexpr int kDwords = 2 * F::kBytes / 4;                 // raw dwords per row: 9 or 17
    static constexpr int kBDwords = kGemmBN * kDwords;                // ... per tile
    // A weight stage holds two consecutive pairs: row r's 2 kDwords dwords
    // (pair 2Q, then pair 2Q + 1, contiguous in the row) at r * 2 kDwords.
    static constexpr int kBQDwords = 2 * kBDwords;                    // ... per stage
    static constexpr int kBQLoads = (kBQDwords + 255) / 256;          // 4-byte loads per 256 threads
    static constexpr int kBQSlots = kBQLoads * 256;                   // LDS dwords per stage
};

// Ring depths: a pair's activation slab is loaded kA steps before the pair is
// computed; the raw weight bytes go two pairs per stage into kBQ stages, each
// loaded 2 kBQ - 1 steps before its first pair. Measured on MI355X
// (2048 x 14336 x 4096, one process), with one pair per weight stage: Q4_0
// is fastest at 4 activation stages (3 costs 2.5 %), Q8_0, whose four
// activation stages do not fit next to its weight stages, at 3; two pairs
// per weight stage gained about 1 %, and a third weight stage (five steps
// ahead) cost 1-3 % on every form.
// HO ("hi only") selects the bfloat16-activation form: one binary16 term per
// activation (exact, see k_gemm_prep_bf16), so a slab is half the size and a
// tile-block needs one MFMA instead of two. With its 128 x 32 wavefront tiles
// both formats are fastest at 4 activation stages (5 costs 3-4 %; 3 stages of
// its slab would not hold the final reduction).
template <class F, bool HO>
struct RingDepth;
template <>
struct RingDepth<FmtQ4_0, false> {
    static constexpr int kA = 4, kBQ = 2;
};
template <>
struct RingDepth<FmtQ8_0, false> {
    static constexpr int kA = 3, kBQ = 2;
};
template <>
struct RingDepth<FmtQ4_0, true> {
    static constexpr int kA = 4, kBQ = 2;
};
template <>
struct RingDepth<FmtQ8_0, true> {
    static constexpr int kA = 4, kBQ = 2;
};

// 16-byte A operands per (128-row tile, block): hi and lo, or hi only.
template <bool HO>
constexpr int slab_ops() { return HO ? kOpsPerBlockTile / 2 : kOpsPerBlockTile; }

template <class F, bool HO>
struct SplitLds {
    static constexpr int DA = RingDepth<F, HO>::kA, DBQ = RingDepth<F, HO>::kBQ;
    u32x4 a[DA][2 * slab_ops<HO>()];          // a pair's slab: [kg][hl][sub][lane], as in the workspace
    uint32_t b[DBQ][PairGeom<F>::kBQSlots];   // two pairs: [row][2 kDwords]; slots past the tile are never read
};
static_assert(sizeof(SplitLds<FmtQ4_0, false>) <= kLdsBytes &&
                  sizeof(SplitLds<FmtQ8_0, false>) <= kLdsBytes &&
                  sizeof(SplitLds<FmtQ4_0, true>) <= kLdsBytes &&
                  sizeof(SplitLds<FmtQ8_0, true>) <= kLdsBytes,
              "the rings fit in LDS");

// s_waitcnt immediates (gfx9 encoding): vmcnt(n) lgkmcnt(0), expcnt unchanged.
constexpr int waitcnt_vm_lgkm0(int n) { return (n & 15) | ((n >> 4) << 14) | 0x70; }

// Wait until this wavefront has at most `vm` vector-memory operations
// outstanding and all its LDS operations are done, then meet the workgroup.
// A raw s_barrier: __syncthreads() would also wait for every outstanding
// direct-to-LDS load, which are meant to stay in flight. The empty asm
// statements keep the compiler from moving LDS accesses across it.
template <int VM>
__device__ __forceinline__ void ring_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(VM));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Loads a loading wavefront may still have in flight at the barrier that ends
// step p (parity par) of k_gemm_split's ring, when pair p + 2 must be
// complete: step s issues na A loads (pair s + da) and, for odd s, then nb B
// loads (pairs s + lb and s + lb + 1), in that order; a load is identified by
// (step, slot), and the count is the loads after the last one pair p + 2 needs.
constexpr int ring_in_flight(int par, int da, int lb, int na, int nb)
{
    const int p = 1000 + par, q = p + 2;
    const int a_step = q - da, a_slot = na - 1;
    const int b_step = 2 * (q / 2) - lb, b_slot = na + nb - 1;
    int ls = a_step, lk = a_slot;
    if (b_step > ls || (b_step == ls && b_slot > lk))
        ls = b_step, lk = b_slot;
    int n = 0;
    for (int st = ls; st <= p; ++st) {
        const int slots = na + ((st & 1) ? nb : 0);
        for (int k = 0; k < slots; ++k)
            if (st > ls || k > lk)
                ++n;
    }
    return n;
}

// In row_exp, GROUPED: a tile row whose row of y another one stores.
constexpr int kNotStored = INT_MIN;

// One K segment of the product: ahl points at the operands of block kb0 of
// the first row tile (a row tile holds nblk_row blocks of operands) and w at
// block kb0 of weight row 0 (a weight row is nblk_row blocks); the segment
// spans nblk blocks (even). row_exp: per-row exponents of the activation
// operands, undone on the result rows (always for the bfloat16 form, HO; for
// the two-term form when not null). accumulate: add the segment's result to y.
// GROUPED: the row tiles are those of the groups, each padded to whole tiles,
// in the operands and in row_exp; group e multiplies the e-th weight matrix,
// and row r of y is the one that the group's list names (none for the
// padding). RMH: row subtiles that the hi-only form computes (the tile's rows
// past 16 RMH, of which a group's last tile can have many, are not there).
template <class F, bool HO, bool GROUPED, int RMH = 8>
__device__ __forceinline__ void gemm_split_body(
    const u32x4 *__restrict__ ahl, const uint8_t *__restrict__ w, float *__restrict__ y, int M,
    int N, int nblk_row, int nblk, int tiles_m, int tiles_n, const int *__restrict__ row_exp,
    int accumulate, const Groups &gr, const GroupTile &gt, SplitLds<F, HO> &lds)
{
    using G = PairGeom<F>;
    // MFMA tiles per wavefront: the hi-only form takes 128 rows x 32 columns
    // (8 x 2), so no two wavefronts of a K group decode the same weight
    // columns; the two-term form keeps 64 x 64 (4 x 4), which leaves room for
    // its lo operands in registers.
    constexpr int RM = HO ? RMH : 4, CN = HO ? 2 : 4;
    constexpr int SO = slab_ops<HO>();           // A operands per (tile, block)
    // A loads (1 KB each) per pair in eighths of the workgroup (the four
    // loading wavefronts issue twice these).
    constexpr int NA = 2 * SO / (8 * 64);
    constexpr int DA = RingDepth<F, HO>::kA, DBQ = RingDepth<F, HO>::kBQ;
    // Weight stages are loaded LB = 2 DBQ - 1 steps ahead of their first pair;
    // the first PRO steps' loads precede the first pair.
    constexpr int LB = 2 * DBQ - 1, PRO = DA > LB ? DA : LB;
    static_assert(DA >= 3 && DBQ >= 2, "ring depths");

    int mt, m0, n0;
    [[maybe_unused]] int pos0 = 0, pos1 = 0;   // GROUPED: the tile's positions
    if constexpr (GROUPED) {
        mt = gt.before + gt.mt, m0 = mt * kGemmBM, n0 = gt.nt * kGemmBN;
        pos0 = gt.lo + gt.mt * kGemmBM, pos1 = gt.hi;
        w += (size_t)gt.e * (size_t)N * ((size_t)nblk_row * F::kBytes);
    } else {
        const int T = tiles_m * tiles_n, L = blockIdx.x;
        const int t = (T % 8 == 0) ? (L % 8) * (T / 8) + L / 8 : L;
        mt = t / tiles_n, m0 = mt * kGemmBM, n0 = (t % tiles_n) * kGemmBN;
    }

    const int tid = threadIdx.x, lane = tid & 63;
    // The wavefront index, made visibly uniform so that branches on it are scalar.
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kg = wave >> 2, wm = HO ? 0 : (wave >> 1) & 1, wn = HO ? (wave & 3) : (wave & 1);
    const int li = lane & 15, g = lane >> 4;
    const int npairs = nblk >> 1;
    const uint32_t magic_v = magic_vgpr<F>();
    const size_t row_bytes = (size_t)nblk_row * F::kBytes;

    // Direct-to-LDS loads, issued by the four wavefronts of K group 0 only
    // (the same count on each, so their vmcnt moves in the same steps; K group
    // 1 issues none and computes through the loads' issue stalls: 2-3% faster
    // than spreading the loads over all eight), as buffer loads: one buffer
    // resource per operand for the workgroup's tile, a fixed per-lane offset
    // and a per-pair scalar offset, so the step's addressing is scalar work.
    // A, per pair: 2 NA (8, or 4 hi-only) 16-byte loads, 1 KB each, at entries
    // (2 NA lw + i) * 64 + lane of the slab (lw = wave % 4), whose workspace
    // order is the LDS order. B, per two pairs (every other step): NBQ 4-byte
    // loads at dword slots j * 64 + lane, j = lw + 4 r; slot t < 128 2 kDwords
    // is dword t % (2 kDwords) of the two pairs' bytes of row t / (2 kDwords),
    // higher slots re-read a valid dword into unused LDS. Two pairs per load
    // instruction put each row's 72 (or 136) contiguous bytes in one
    // instruction instead of 36 (68) in each of two: a quarter fewer weight
    // loads (9 against 12 per two Q4_0 pairs, less padding), about 1% faster.
    // The ranges of both resources fit 32 bits (K <= 2^22 on this path); each
    // ends with the segment's last block.
    const __amdgpu_buffer_rsrc_t arsrc = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(ahl + (size_t)mt * nblk_row * SO), (short)0, (int)((uint32_t)nblk * SO * 16u),
        kBufferRsrcWord3);
    const int brows = min(kGemmBN, N - n0);
    const __amdgpu_buffer_rsrc_t brsrc = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(w + (size_t)n0 * row_bytes), (short)0,
        (int)((brows - 1) * row_bytes + (size_t)nblk * F::kBytes), kBufferRsrcWord3);
    // Loads of a loading wavefront: NA2 A loads per pair, NBQ B loads per
    // two pairs.
    constexpr int NA2 = 2 * NA, NBQ = G::kBQLoads;
    constexpr int kDQ = 2 * G::kDwords;             // B dwords per row and stage
    const int lw = wave & 3;
    const uint32_t a_voff = (uint32_t)((lw * NA2 * 64 + lane) * 16);
    uint32_t b_voff[NBQ];
#pragma unroll
    for (int r = 0; r < NBQ; ++r) {
        const int tt = min((lw + 4 * r) * 64 + lane, G::kBQDwords - 1);
        const int row = tt / kDQ, dw = tt % kDQ;
        b_voff[r] = (uint32_t)(min(row, brows - 1) * (int)row_bytes + 4 * dw);
    }
    // Load k of a step on a loading wavefront: the NA2 A loads of pair pa,
    // then (odd steps) the NBQ B loads of pairs 2 qb and 2 qb + 1 (k is a
    // compile-time constant where this is called).
    auto issue_load = [&](int pa, int qb, int k) __attribute__((always_inline)) {
        if (k < NA2)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                arsrc, (__attribute__((address_space(3))) void *)(lds.a[pa % DA] + (lw * NA2 + k) * 64),
                16, a_voff + k * 1024, (int)((uint32_t)pa * (2u * SO * 16u)), 0, 0);
        else
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                brsrc, (__attribute__((address_space(3))) void *)(lds.b[(unsigned)qb % DBQ] + (lw + 4 * (k - NA2)) * 64),
                4, b_voff[k - NA2], qb * (4 * F::kBytes), 0, 0);
    };

    f32x4 acc[RM][CN];
#pragma unroll
    for (int ms = 0; ms < RM; ++ms)
#pragma unroll
        for (int ns = 0; ns < CN; ++ns)
            acc[ms][ns] = (f32x4){0.f, 0.f, 0.f, 0.f};
    const f32x4 zero4 = {0.f, 0.f, 0.f, 0.f};
    const f16 sc = (f16)0x1p-11f;
    const f16x8 scale = {sc, sc, sc, sc, sc, sc, sc, sc};

    auto run_group = [&](auto kg_c) __attribute__((always_inline)) {
        constexpr int KG = decltype(kg_c)::value;
        // Loads per step of this wavefront (even steps: A only; odd steps: A
        // and B): all of the workgroup's on K group 0's four, none on K group
        // 1's.
        constexpr int NAK = KG == 0 ? NA2 : 0, NBK = KG == 0 ? NBQ : 0;
        // B of column group ns, block 2p + KG: the row's raw pair bytes hold block
        // KG at byte kBytes KG. KG is a compile-time constant (the loop exists
        // once per K group), so the realignment (where the quant bytes straddle
        // dwords) and the half of the dword that holds d are fixed per loop.
        struct BCol {
            QsRaw<F, KG> qs;
            uint32_t dw;
        };
        auto read_b = [&](const uint32_t *bstage, int ns) __attribute__((always_inline)) {
            const uint32_t *rb = bstage + (wn * (CN * 16) + ns * 16 + li) * kDQ;
            return BCol{read_qs_raw<F, KG>(rb, g), rb[d_dword<F, KG>()]};
        };
        // The operands of one pair held in registers: the A operands of the
        // wavefront's RM row groups and the raw B bytes of its CN column
        // groups.
        struct Ops {
            f16x8 hi[RM], lo[HO ? 1 : RM];
            BCol b[CN];
        };
        // Part i of pair q's operands (row groups i RM/CN .. (i+1) RM/CN - 1,
        // column group i).
        auto read_ops = [&](int q, Ops &o, int i) __attribute__((always_inline)) {
            const u32x4 *ap = lds.a[q % DA] + KG * SO + wm * RM * 64 + lane;
#pragma unroll
            for (int r = i * (RM / CN); r < (i + 1) * (RM / CN); ++r) {
                o.hi[r] = bitcast<f16x8>(ap[r * 64]);
                if constexpr (!HO)
                    o.lo[r] = bitcast<f16x8>(ap[8 * 64 + r * 64]);
            }
            o.b[i] = read_b(lds.b[((unsigned)q >> 1) % DBQ] + (q & 1) * G::kDwords, i);
        };
        // LDS reads of one part.
        constexpr int kDsReads = (RM / CN) * (HO ? 1 : 2) + QsRaw<F, KG>::n + 1;

        // Software pipeline over the four column groups of a pair: the MFMAs of
        // group ns are issued between the scale FMAs of group ns - 1 (whose results
        // are ready) and the decode of group ns + 1. Group results alternate
        // between two register sets by the parity of ns, and the group before
        // group 0 is group 3 of the previous pair (zeros before the first pair),
        // so every index is a compile-time constant.
        f32x4 cbuf[2][RM];
        float dbuf[2] = {0.0f, 0.0f};
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int ms = 0; ms < RM; ++ms)
                cbuf[h][ms] = zero4;
        struct BOps {
            f16x8 q, s;   // the codes (x 2^kHiLog2 in slots 4..7) and the same times 2^-11
            float d;
        };
        auto decode_b = [&](const BCol &bc) __attribute__((always_inline)) {
            uint32_t x[F::kQsDwords];
            align_qs<F, KG>(bc.qs, x);
            BOps o;
            o.d = f16_bits_to_f32(d_from_dword<F, KG>(bc.dw));
            o.q = F::decode(x, magic_v);
            if constexpr (!HO)
                o.s = o.q * scale;
            return o;
        };
        // One scheduling region per column group ns: its eight MFMAs (the four lo
        // products, then the four hi products that add onto them) interleaved
        // with the scale FMAs of group ns - 1, the decode of group ns + 1 and
        // part ns of the next pair's operands (LDS reads that land during this
        // pair's MFMAs, so no step starts by waiting on LDS). The scheduling-group
        // barriers ask for one MFMA, one LDS read while any remain, then four VALU
        // instructions, eight times per region; hard barriers between regions
        // keep that order.
        auto compute_pair = [&](auto odd_c, const Ops &cur_ops, Ops &next_ops, int next_pair,
                                int dma_a, int dma_b) __attribute__((always_inline)) {
            constexpr int NLK = NAK + (decltype(odd_c)::value ? NBK : 0);
            BOps cur = decode_b(cur_ops.b[0]);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int ns = 0; ns < CN; ++ns) {
                f32x4 *c = cbuf[ns & 1];
                const f32x4 *cp = cbuf[(ns + 1) & 1];      // group ns - 1 (mod CN; CN is even)
                const float dp = dbuf[(ns + 1) & 1];
                // The two-term form multiplies the small lo terms first and adds
                // the hi products onto them (the rounding of the lo chain then
                // acts on sums 2^-11 the size of the hi ones).
#pragma unroll
                for (int ms = 0; ms < RM; ++ms) {
                    if constexpr (HO)
                        c[ms] = __builtin_amdgcn_mfma_f32_16x16x32_f16(cur_ops.hi[ms], cur.q, zero4, 0, 0, 0);
                    else
                        c[ms] = __builtin_amdgcn_mfma_f32_16x16x32_f16(cur_ops.lo[ms], cur.s, zero4, 0, 0, 0);
                }
                read_ops(next_pair, next_ops, ns);
                // The step's loads go out spread over the four regions (loads
                // [NLK ns / 4, NLK (ns + 1) / 4), rounded up) and, within a region,
                // between MFMAs, so the address unit works while the matrix cores
                // do and no wavefront's MFMAs queue behind a load. They write LDS,
                // so they follow this region's LDS reads in program order (the
                // compiler keeps LDS accesses it cannot tell apart in order).
#pragma unroll
                for (int k = (NLK * ns + CN - 1) / CN; k < (NLK * (ns + 1) + CN - 1) / CN; ++k)
                    issue_load(dma_a, dma_b, k);
                const int np = (ns + CN - 1) % CN;
#pragma unroll
                for (int ms = 0; ms < RM; ++ms)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        acc[ms][np][q] = fmaf(dp, cp[ms][q], acc[ms][np][q]);
                // Pin these FMAs to this region: IR passes would otherwise sink
                // them past the scheduling barriers, to the end of the pair.
                if constexpr (RM == 2)
                    asm volatile("" : "+v"(acc[0][np]), "+v"(acc[1][np]));
                else if constexpr (RM == 4)
                    asm volatile("" : "+v"(acc[0][np]), "+v"(acc[1][np]), "+v"(acc[2][np]), "+v"(acc[3][np]));
                else
                    asm volatile("" : "+v"(acc[0][np]), "+v"(acc[1][np]), "+v"(acc[2][np]), "+v"(acc[3][np]),
                                      "+v"(acc[4][np]), "+v"(acc[5][np]), "+v"(acc[6][np]), "+v"(acc[7][np]));
                BOps nxt = cur;
                if (ns + 1 < CN)
                    nxt = decode_b(cur_ops.b[ns + 1]);
                if constexpr (!HO) {
#pragma unroll
                    for (int ms = 0; ms < RM; ++ms)
                        c[ms] = __builtin_amdgcn_mfma_f32_16x16x32_f16(cur_ops.hi[ms], cur.q, c[ms], 0, 0, 0);
                }
                dbuf[ns & 1] = cur.d;
                // Eight MFMAs per region, each followed by LDS reads while any
                // remain, the region's loads towards its end, and its share of
                // the VALU work.
                constexpr int NM = RM * (HO ? 1 : 2);
                constexpr int kDsPerSlot = (kDsReads + NM - 1) / NM;
                constexpr int kValuPerSlot = HO ? (F::kBytes == kQ4Bytes ? 4 + 24 / RM : 4 + 16 / RM) : 4;
                constexpr int kRegionLoads = (NLK + CN - 1) / CN;   // at most, per region
                const int nl = (NLK * (ns + 1) + CN - 1) / CN - (NLK * ns + CN - 1) / CN;
#pragma unroll
                for (int u = 0; u < NM; ++u) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // one MFMA
                    if (u * kDsPerSlot < kDsReads)
                        __builtin_amdgcn_sched_group_barrier(0x100, kDsPerSlot, 0);   // LDS reads
                    if (u >= NM - nl && u >= NM - kRegionLoads)
                        __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);   // one load
                    __builtin_amdgcn_sched_group_barrier(0x002, kValuPerSlot, 0);   // VALU
                }
                __builtin_amdgcn_sched_barrier(0);
                cur = nxt;
            }
        };

        // Ring schedule: step p issues the A loads of pair p + DA and, when p is
        // odd, then the B loads of pairs p + LB and p + LB + 1 (double stage
        // Q = (p + LB) / 2, in B stage Q % DBQ). Pair q's A slab goes to A
        // stage q % DA during step q - DA, its B bytes to B stage (q / 2) % DBQ
        // during step 2 (q / 2) - LB (q - LB or q - LB - 1). Both are complete
        // by the barrier ending step q - 2, are read into registers during
        // step q - 1, and pair q is computed in step q. An A stage is loaded
        // again in step q (pair q + DA), after the barrier that ends step
        // q - 1, by which every wavefront has read it; B stage Q % DBQ again
        // in step 2 Q + 1, after the barrier ending step 2 Q, by which pair
        // 2 Q + 1's bytes are read. Loads complete in issue order, so at the
        // barrier ending step p the loads issued after the last one pair p + 2
        // needs may still be in flight: ring_in_flight counts them, one count
        // for even and one for odd p (near the end, where fewer are issued, the
        // barrier waits for everything). What the last step reads is discarded;
        // the loads that it leaves in flight are waited for before the epilogue.
        constexpr int kInFlightEven = ring_in_flight(0, DA, LB, NAK, NBK);
        constexpr int kInFlightOdd = ring_in_flight(1, DA, LB, NAK, NBK);
        static_assert(kInFlightEven < 64 && kInFlightOdd < 64, "vmcnt counts to 63");
        // The loads of steps -PRO .. -1, in the order those steps would issue
        // them (a step before the first A load issues only its B loads). A step whose
        // pair is past the last one reloads the last pair (or two) into its own
        // stage (the same bytes), so every step issues its count of loads and,
        // with at least PRO pairs, every barrier can count them; shorter problems
        // wait for all. K group 1 has no loads of its own in flight: its
        // barriers only order, and wait for the loaders, which wait for theirs
        // before the barrier.
        const bool counted = npairs >= PRO;
        const int last = npairs - 1, lastq = last >> 1;
        for (int t = -PRO; t < 0; ++t) {
#pragma unroll
            for (int k = 0; k < NAK + NBK; ++k)
                if (k < NAK ? t + DA >= 0 : (t & 1) != 0)
                    issue_load(min(t + DA, last), min((t + LB) / 2, lastq), k);
        }
        if (counted)
            ring_barrier<kInFlightOdd>();   // pairs 0 and 1 complete
        else
            ring_barrier<0>();
        Ops O0, O1;
#pragma unroll
        for (int i = 0; i < CN; ++i)
            read_ops(0, O0, i);
        // Step 0 reloads A stage 0: every wavefront must have read pair 0's
        // operands first.
        if (counted)
            ring_barrier<kInFlightOdd>();
        else
            ring_barrier<0>();
        auto step = [&](auto odd_c, int p, const Ops &cur_ops, Ops &next_ops) __attribute__((always_inline)) {
            constexpr bool odd = decltype(odd_c)::value;
            compute_pair(odd_c, cur_ops, next_ops, p + 1, min(p + DA, last), min((p + LB) / 2, lastq));
            if (counted)
                ring_barrier<odd ? kInFlightOdd : kInFlightEven>();   // pair p + 2 complete
            else
                ring_barrier<0>();
        };
        for (int p = 0; p < npairs; p += 2) {
            step(std::false_type{}, p, O0, O1);
            if (p + 1 < npairs)
                step(std::true_type{}, p + 1, O1, O0);
        }
        // FMAs of the last column group (group CN - 1 of the last pair, in set 1).
#pragma unroll
        for (int ms = 0; ms < RM; ++ms)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                acc[ms][CN - 1][q] = fmaf(dbuf[1], cbuf[1][ms][q], acc[ms][CN - 1][q]);
    };
    if (kg == 0)
        run_group(std::integral_constant<int, 0>{});
    else
        run_group(std::integral_constant<int, 1>{});

    // The last steps' reloads may still be on their way (a counted barrier
    // leaves them in flight, and K group 1, which issued none, cannot wait for
    // them): they land before any of the rings' LDS is written below.
    ring_barrier<0>();

    // Group 1 hands its partial tile to group 0 through LDS:
    // [wavefront of the group][value][lane].
    float *red = reinterpret_cast<float *>(&lds.a[0][0]);
    static_assert(sizeof(lds.a) >= 4 * 64 * 64 * sizeof(float), "reduction buffer");
    const int wq = wave & 3;
    if (kg == 1) {
#pragma unroll
        for (int ms = 0; ms < RM; ++ms)
#pragma unroll
            for (int ns = 0; ns < CN; ++ns)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    red[(wq * 64 + ms * (CN * 4) + ns * 4 + q) * 64 + lane] = acc[ms][ns][q];
    }
    // GROUPED: the tile's rows of y and their exponents, fetched at once (2048
    // tokens, 2 of 8 experts, 14336 x 4096, Q4_0 with bfloat16: 832 us when each
    // is read as its row is stored, 780 so).
    [[maybe_unused]] int2 *rows = reinterpret_cast<int2 *>(&lds.b[0][0]);
    if constexpr (GROUPED) {
        static_assert(sizeof(lds.b) >= kGemmBM * sizeof(int2), "a row and an exponent each");
        const int r = tid - kSplitGemmThreads / 2;
        if (r >= 0 && r < kGemmBM)
            rows[r] = pos0 + r < pos1 && row_exp[m0 + r] != kNotStored
                          ? int2{group_row(gr, pos0 + r), row_exp[m0 + r]} : int2{-1, 0};
    }
    __syncthreads();
    if (kg == 0) {
        // Lane (li, g) of tile (ms, ns) holds rows 4g..4g+3 of column li.
        // Offsets are 32-bit (M N < 2^31 on this path, checked at launch).
        // Rows of scaled activations (every form that passes row exponents)
        // are scaled back by 2^-row_exp[m]; a later K segment adds its part to
        // what the earlier ones left in y.
        const bool scaled_rows = HO || row_exp != nullptr;
        const int mb = m0 + wm * (RM * 16) + 4 * g, nb = n0 + wn * (CN * 16) + li;
#pragma unroll
        for (int ms = 0; ms < RM; ++ms) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int m = mb + ms * 16 + q;
                if constexpr (GROUPED) {
                    const int2 to = rows[m - m0];
                    if (to.x < 0)
                        continue;
                    const int pe = to.y;
                    float *yr = y + (size_t)to.x * (size_t)N + nb;
#pragma unroll
                    for (int ns = 0; ns < CN; ++ns) {
                        float v = acc[ms][ns][q] + red[(wq * 64 + ms * (CN * 4) + ns * 4 + q) * 64 + lane];
                        v = ldexpf(v, -pe);
                        if (nb + ns * 16 < N)
                            yr[ns * 16] = accumulate ? yr[ns * 16] + v : v;
                    }
                    continue;
                }
                const uint32_t row_off = (uint32_t)m * (uint32_t)N + (uint32_t)nb;
                int pe = 0;
                if (scaled_rows && m < M)
                    pe = row_exp[m];
#pragma unroll
                for (int ns = 0; ns < CN; ++ns) {
                    float v = acc[ms][ns][q] + red[(wq * 64 + ms * (CN * 4) + ns * 4 + q) * 64 + lane];
                    if (scaled_rows)
                        v = ldexpf(v, -pe);
                    if (m < M && nb + ns * 16 < N) {
                        if (accumulate)
                            v += y[row_off + ns * 16];
                        y[row_off + ns * 16] = v;
                    }
                }
            }
        }
    }
}

template <class F, bool HO>
__global__ __launch_bounds__(kSplitGemmThreads) void k_gemm_split(
    const u32x4 *__restrict__ ahl, const uint8_t *__restrict__ w, float *__restrict__ y, int M,
    int N, int nblk_row, int nblk, int tiles_m, int tiles_n, const int *__restrict__ row_exp,
    int accumulate)
{
    __shared__ SplitLds<F, HO> lds;
    gemm_split_body<F, HO, false>(ahl, w, y, M, N, nblk_row, nblk, tiles_m, tiles_n, row_exp,
                                  accumulate, Groups{nullptr, nullptr, 0, 0, 1, 0},
                                  GroupTile{0, 0, 0, 0, 0, 0}, lds);
}

__device__ __forceinline__ float bf16_bits_to_f32(uint32_t bits) { return __uint_as_float(bits << 16); }

// Largest |a| of row `row` (K bfloat16 values, K % 32 == 0) as a cleared-sign
// bit pattern, in every lane of the wavefront.
__device__ __forceinline__ uint32_t row_max_bits_bf16(const uint16_t *__restrict__ row, int K,
                                                      int lane)
{
    // A row is a whole number of 64-byte lines, read 16 bytes a lane.
    const uint4 *r4 = reinterpret_cast<const uint4 *>(row);
    uint32_t mx = 0;
#pragma unroll 8
    for (int i = lane; i < K / 8; i += 64) {
        const uint4 v = r4[i];
        const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            mx = max(mx, max(w4[j] & 0x7FFFu, (w4[j] >> 16) & 0x7FFFu));
    }
    return wave_max_u32(mx);
}

// p = 15 - E for a largest magnitude in [2^E, 2^(E+1)); 0 for zero or non-finite.
__device__ __forceinline__ int row_exp_from_bits(uint32_t mx)
{
    if (mx == 0 || mx >= 0x7F80u)
        return 0;
    const int ef = (int)(mx >> 7);
    // Subnormals are (mantissa) 2^-133.
    const int E = ef > 0 ? ef - 127 : (31 - __builtin_clz(mx)) - 133;
    return 15 - E;
}

// Largest |a| of row `row` (K f32 values, K % 32 == 0, 16-byte aligned) as a
// cleared-sign bit pattern, in every lane of the wavefront. Sixteen 16-byte
// loads per lane per round are issued before any is used (a 4096-element row
// in one round), so a compute unit keeps enough bytes in flight even with one
// wavefront per row.
__device__ __forceinline__ uint32_t row_max_bits_f32(const float *__restrict__ row, int K, int lane)
{
    const uint4 *r4 = reinterpret_cast<const uint4 *>(row);
    uint32_t mx = 0;
#pragma unroll 16
    for (int i = lane; i < K / 4; i += 64) {
        const uint4 v = r4[i];
        mx = max(mx, max(max(v.x & 0x7FFFFFFFu, v.y & 0x7FFFFFFFu),
                         max(v.z & 0x7FFFFFFFu, v.w & 0x7FFFFFFFu)));
    }
    return wave_max_u32(mx);
}

// The row's power of two from its largest cleared-sign bit pattern.
__device__ __forceinline__ int row_exp_from_bits_f32(uint32_t mx)
{
    int p = 0;
    if (mx != 0 && mx < 0x7F800000u) {
        const int ef = (int)(mx >> 23);
        // Subnormals are (mantissa) 2^-149.
        const int E = ef > 0 ? ef - 127 : (31 - __builtin_clz(mx)) - 149;
        p = 14 - E;
    }
    return p;
}

// Longest run of block partials that one accumulator adds in sequence in a
// launch. Longer K is cut into segments, one launch each, every launch after
// the first adding its part into y; see the summation order at the top.
constexpr int kMaxChain = 112;

struct KSegments {
    int n, len;   // n segments of len blocks (the last one the rest)
};

// per_term: blocks per term of an accumulator's chain, 2 on the split kernel
// (its two K groups take alternate blocks), 1 on the general kernel.
inline KSegments k_segments(int nblk, int per_term)
{
    const int terms = (nblk + per_term - 1) / per_term;
    const int n = (terms + kMaxChain - 1) / kMaxChain;
    const int len = (terms + n - 1) / n * per_term;
    return {(nblk + len - 1) / len, len};
}

}  // namespace q4k
