// The decode GEMV's streaming kernel, for the GEMV (gemv.hip) and the products
// grouped by expert (grouped.hip).
#pragma once

#include <type_traits>
#include <utility>

#include "device_common.h"
#include "formats.h"

namespace q4k {

constexpr int kGemvStreamWaves = 8;

// Split v into binary16 hi + lo with hi = f16(v) and lo = f16(v - hi).
__device__ __forceinline__ void split2(float v, f16 &hi, f16 &lo)
{
    hi = (f16)v;
    lo = (f16)(v - (float)hi);
}

// split2 of x0 sc and x1 sc (sc a power of two, so x sc is exact), packed:
// hi = (f16(x0 sc), f16(x1 sc)) and lo = (f16(x0 sc - hi0), f16(x1 sc - hi1)).
// Each half is one mixed-precision FMA (f32 operands, f16 result, one
// rounding), and lo reads its hi half straight from the packed register.
__device__ __forceinline__ void split2_pair(float x0, float x1, float sc, uint32_t &hi,
                                            uint32_t &lo)
{
    uint32_t h, l;
    asm("v_fma_mixlo_f16 %0, %1, %2, 0" : "=v"(h) : "v"(x0), "v"(sc));
    asm("v_fma_mixhi_f16 %0, %1, %2, 0" : "+v"(h) : "v"(x1), "v"(sc));
    asm("v_fma_mixlo_f16 %0, %1, %2, -%3 op_sel_hi:[0,0,1]" : "=v"(l) : "v"(x0), "v"(sc), "v"(h));
    asm("v_fma_mixhi_f16 %0, %1, %2, -%3 op_sel:[0,0,1] op_sel_hi:[0,0,1]"
        : "+v"(l) : "v"(x1), "v"(sc), "v"(h));
    hi = h;
    lo = l;
}

// max(m, |a|, |b|) for m >= 0, one instruction: the absolute values are
// operand modifiers, and in inline asm the compiler adds no canonicalizing
// of the loaded values (as it would for fmaxf). For finite values the result
// equals the largest cleared-sign bit pattern; only loaded activations and
// the running maximum are read (no result of an in-flight MFMA).
__device__ __forceinline__ float max3_abs(float m, float a, float b)
{
    float r;
    asm("v_max3_f32 %0, %1, |%2|, |%3|" : "=v"(r) : "v"(m), "v"(a), "v"(b));
    return r;
}

// Largest A value of a row is 2^kHiLog2 max|a| 2^p: p puts it in [2^14, 2^15).
template <class F>
__device__ __forceinline__ int row_scale_exp(float am)
{
    int e = 0;
    frexpf(am, &e);                                  // am in [2^(e-1), 2^e)
    const int p = (am == 0.0f) ? 0 : 15 - F::kHiLog2 - e;
    return p > 120 ? 120 : (p < -120 ? -120 : p);
}

// bfloat16 activations (BF): a bfloat16 value has an 8-bit significand, so
// after a power-of-two scale that puts the largest A value of its row in
// [2^15, 2^16) every element within 2^28 (Q4_0) or 2^32 (Q8_0) of the row's
// largest magnitude is exactly a binary16 number. One A row per activation
// row then replaces the hi / lo pair: A row m is activation row m, and lane
// (j, g) accumulates C rows 4g..4g+3, activation rows 4g + r.
template <class F>
__device__ __forceinline__ int row_scale_exp_bf16(float am)
{
    int e = 0;
    frexpf(am, &e);                                  // am in [2^(e-1), 2^e)
    return (am == 0.0f || !(am <= 3.4e38f)) ? 0 : 16 - F::kHiLog2 - e;
}

__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

template <bool BF, int M>
struct GemvRows {
    static constexpr int NI = BF ? M : 2 * M;                              // A rows in use
    static constexpr int NACC = BF ? (M < 4 ? M : 4) : (M == 1 ? 2 : 4);   // C rows a lane owns
    static constexpr int NOUT = BF ? NACC : NACC / 2;                      // activation rows a lane owns
    // Activation row of a lane's output h (lane group g).
    static __device__ __forceinline__ int row(int g, int h) { return BF ? 4 * g + h : 2 * g + h; }
};

// ---------------------------------------------------------------------------
// Streaming variant for rows that are 16-byte aligned (K % 256 == 0), which
// covers the decode shapes. Same arithmetic as above; what changes is how the
// weight bytes reach the matrix cores:
// * Each wavefront owns a run of blocks of the workgroup's 16 rows and walks it
//   in chunks of CH blocks (CH * 18 or CH * 34 bytes per row, a multiple of
//   16 for CH = 8 or 16). A chunk is fetched with aligned 16-byte loads, lane (r, c) taking
//   16-byte column c of row r, and written unchanged into the wavefront's own
//   LDS area. Operands are then read back with aligned LDS dword pairs and
//   realigned with v_alignbyte. No global load is narrower than 16 bytes or
//   misaligned, and the next chunk's loads are in flight while the current
//   one is computed.
// * The activations of a chunk are split by the whole wavefront (each lane a
//   few 8-element groups) and passed to the A-operand lanes through LDS. The
//   power-of-two scale is chosen per (chunk, activation row) from the chunk's
//   own max |a|, and undone on that chunk's f32 partial, so no workgroup-wide
//   pass over the activations is needed.
// * Wavefront partials meet in LDS once, at the end, and are summed in a
//   fixed order.

// Order LDS traffic between the lanes of one wavefront: its LDS operations
// execute in issue order, so it is enough that the compiler keeps them there.
__device__ __forceinline__ void wave_lds_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <class F, int M, int NW, int CH_, bool BF, int RPW_ = 16, bool LA_ = false>
struct GemvStreamCfg {
    static constexpr int CH = CH_;                        // blocks per chunk (8 or 16)
    static constexpr int RPW = RPW_;                      // weight rows per workgroup (16 or 8)
    // LA (line-aligned loads; rows a whole number of 128-byte lines from a
    // line-aligned base): a chunk row is fetched as the NLN whole lines that
    // hold it. A chunk starts at a multiple of its byte count, so its offset
    // into its first line is a multiple of that count's lowest set bit, at
    // most kMaxShift; from every such offset it spans exactly NLN lines
    // (asserted), so the lines never pass the end of the row.
    static constexpr bool LA = LA_;
    static constexpr int kChunkBytes = CH * F::kBytes;
    static constexpr int kMaxShift = (kChunkBytes & 127) == 0 ? 0 : 128 - (kChunkBytes & -kChunkBytes);
    static constexpr int NLN = (kMaxShift + kChunkBytes + 127) / 128;
    static_assert(!LA || (kChunkBytes + 127) / 128 == NLN,
                  "a chunk spans the same number of lines from every start offset");
    static constexpr int CPR = LA ? 8 * NLN : CH * F::kBytes / 16;   // 16-byte columns per staged row
    // Weight loads: eight lanes per row take 128 contiguous bytes (one cache
    // line's worth), eight rows per load: loads (RPW / 8) c + h cover columns
    // 8c..8c+7 of rows 8h..8h+7, for each of the NG whole groups of eight
    // columns; one more load covers the TC tail columns of all RPW rows
    // (TLPR = 64 / RPW lanes per row).
    static constexpr int NG = CPR / 8, TC = CPR % 8, RH = RPW / 8, TLPR = 64 / RPW;
    static constexpr int NLOAD = RH * NG + (TC > 0 ? 1 : 0);   // 16-byte loads per lane per chunk
    static constexpr int RS = 16 * CPR + 16;              // LDS bytes per staged row
    static constexpr int WBYTES = RPW * RS;               // staged weight bytes per wavefront
    static constexpr int NI = GemvRows<BF, M>::NI;        // A rows in use
    // The A operands of a chunk pass through LDS in AH halves when a whole
    // chunk's would not fit (16 blocks of more than eight A rows).
    static constexpr int AH = (CH == 16 && NI > 8) ? 2 : 1;
    static constexpr int CHH = CH / AH;                   // blocks per A pass
    static constexpr int ABYTES = CHH * 4 * NI * 16;      // A operands per wavefront
    // Activation split: lane l handles activation row l / QN (QN = 64 / MP,
    // MP = M rounded up to a power of two) and, in each A pass, the 8-element
    // groups l % QN + QN r (r < EPP) of that pass's 4 CHH (block, lane group)
    // pairs, so consecutive lanes read consecutive activations.
    static constexpr int MP = M <= 1 ? 1 : (M <= 2 ? 2 : (M <= 4 ? 4 : 8));
    static constexpr int QN = 64 / MP;                    // lanes per activation row
    static constexpr int EPP = (4 * CHH + QN - 1) / QN;   // groups per lane per A pass
    static constexpr int EPL = AH * EPP;                  // ... per chunk
    static constexpr int LDS_PER_WAVE = WBYTES + ABYTES;
    static constexpr int NPART = CH == 16 ? 4 : 2;        // parts a chunk is contracted in
    // Loads (per lane) that hold every byte of the chunk's first b blocks.
    static constexpr int cols_for(int b) { return (F::kBytes * b + 15) / 16; }
    // LA: the lines that hold them at the largest start offset.
    static constexpr int loads_for(int b)
    {
        if constexpr (LA)
            return b == 0 ? 0 : RH * min_c((kMaxShift + F::kBytes * b + 127) / 128, NLN);
        return b == 0 ? 0 : (cols_for(b) <= 8 * NG ? RH * ((cols_for(b) + 7) / 8) : NLOAD);
    }
    static constexpr int min_c(int x, int y) { return x < y ? x : y; }
    static_assert(RPW == 8 || RPW == 16, "eight or sixteen weight rows per workgroup");
    static_assert(TC <= TLPR, "the tail columns fit the lanes of a row");
    static_assert(CH == 8 || CH == 16, "chunks are 8 or 16 blocks");
    static_assert((CH * F::kBytes) % 16 == 0, "a chunk row is whole 16-byte columns");
};

// Calls f(integral_constant<int, P>) for P = 0 .. NP-1, in order.
template <int NP, class F, int... P>
__device__ __forceinline__ void for_each_part_impl(F &&f, std::integer_sequence<int, P...>)
{
    (f(std::integral_constant<int, P>{}), ...);
}
template <int NP, class F>
__device__ __forceinline__ void for_each_part(F &&f)
{
    for_each_part_impl<NP>(f, std::make_integer_sequence<int, NP>{});
}

// Maximum of a non-negative float over the wavefront, returned to every lane.
// Non-negative IEEE floats order like their bit patterns, so the reduction
// runs on integers: DPP within quads, half-rows and rows, then one readlane
// per row of 16 lanes.
__device__ __forceinline__ float wave_max_nonneg(float v)
{
    int x = __builtin_bit_cast(int, v);
    x = max(x, __builtin_amdgcn_mov_dpp(x, 0xB1, 0xF, 0xF, false));    // quad_perm 1,0,3,2
    x = max(x, __builtin_amdgcn_mov_dpp(x, 0x4E, 0xF, 0xF, false));    // quad_perm 2,3,0,1
    x = max(x, __builtin_amdgcn_mov_dpp(x, 0x141, 0xF, 0xF, false));   // row_half_mirror
    x = max(x, __builtin_amdgcn_mov_dpp(x, 0x140, 0xF, 0xF, false));   // row_mirror
    const int r = max(max(__builtin_amdgcn_readlane(x, 0), __builtin_amdgcn_readlane(x, 16)),
                      max(__builtin_amdgcn_readlane(x, 32), __builtin_amdgcn_readlane(x, 48)));
    return __builtin_bit_cast(float, r);
}

// Maximum of a non-negative float over each run of QN consecutive lanes (QN
// = 8, 16, 32 or 64), returned to each lane of the run: DPP within quads,
// half-rows and rows, then across rows.
template <int QN>
__device__ __forceinline__ float lane_run_max_nonneg(float v)
{
    static_assert(QN == 8 || QN == 16 || QN == 32 || QN == 64, "runs of 8, 16, 32 or 64 lanes");
    if constexpr (QN == 64) {
        return wave_max_nonneg(v);
    } else {
        int x = __builtin_bit_cast(int, v);
        x = max(x, __builtin_amdgcn_mov_dpp(x, 0xB1, 0xF, 0xF, false));    // quad_perm 1,0,3,2
        x = max(x, __builtin_amdgcn_mov_dpp(x, 0x4E, 0xF, 0xF, false));    // quad_perm 2,3,0,1
        x = max(x, __builtin_amdgcn_mov_dpp(x, 0x141, 0xF, 0xF, false));   // row_half_mirror
        if constexpr (QN >= 16)
            x = max(x, __builtin_amdgcn_mov_dpp(x, 0x140, 0xF, 0xF, false));   // row_mirror
        if constexpr (QN >= 32)
            x = max(x, __shfl_xor(x, 16));
        return __builtin_bit_cast(float, x);
    }
}

// A operand (block b, lane group g, A row i) sits in LDS at slot
// b ASTRIDE / 16 + g NI + (i ^ a_swz<NI>(b, g)). A write instruction of the
// activation split has eight consecutive lanes on one A row (or hi / lo
// pair) of two consecutive blocks times the four lane groups; unswizzled,
// NI a multiple of 8 puts all eight in one bank group. The XOR, below NI,
// gives each of the eight its own 16-byte bank group, and within one (b, g)
// it only permutes the NI slots, so the operand reads (lane j of group g
// reads row j) stay conflict-free. Other NI keep the plain layout, where the
// conflicts are at most four-way.
template <int NI>
__device__ __forceinline__ int a_swz(int b, int g)
{
    if constexpr (NI == 8 || NI == 16)
        return ((b & 1) << 2) | g;
    else if constexpr (NI == 4)
        return ((b & 1) << 1) | (g >> 1);
    else if constexpr (NI == 2)
        return b & 1;
    else
        return 0;
}

// Calls f(integral_constant<int, B>) for B = B0 .. B1-1, in order.
template <int B0, class F, int... P>
__device__ __forceinline__ void static_for_impl(F &&f, std::integer_sequence<int, P...>)
{
    (f(std::integral_constant<int, B0 + P>{}), ...);
}
template <int B0, int B1, class F>
__device__ __forceinline__ void static_for(F &&f)
{
    static_for_impl<B0>(f, std::make_integer_sequence<int, B1 - B0>{});
}

// NT: the weight loads are non-temporal. With whole-line loads (LA, below) on
// every launch. Otherwise where every wavefront streams one chunk and no
// second workgroup shares its compute unit (about 6% faster at 1 x 4096 x
// 4096 and 8 x 4096 x 4096), and by the row-group loops (LN) from two
// activation rows; with partial lines and more chunks per wavefront or
// workgroups per compute unit it was 3-5% slower.
// MODE 0: as above. MODE 1 (AL): the MFMAs read the chunk's A operands from
// LDS block by block instead of holding all of them in registers (only where
// one pass holds the chunk's A operands, AH == 1). That frees CH * 4 VGPRs, so
// two workgroups share a compute unit and one's loads overlap the other's
// work: taken when there are more workgroups than compute units (and LN,
// below, does not apply) or more than one chunk per wavefront. MODE 2 (PA, f32 activations): `a` holds operands
// prepared once by k_gemv_prep_ops (the two-term A operands of every block in
// [block][lane group][A row] order, then the per-row exponents), loaded
// straight into the A registers: no per-chunk split, scale or LDS pass.
// LN (MODE 0 or 2, one chunk per wavefront, no K split): the workgroup
// walks the row groups blockIdx.x, blockIdx.x + gridDim.x, ... of 16 weight
// rows with the same chunk, so its activations are loaded and split (or its
// prepared operands loaded) once for all of them; once a group's weight bytes
// are staged, the next group's loads are issued, and each group ends with its
// own reduction and store (partials in alternate LDS buffers, one barrier per
// group). Every output sees the same arithmetic as without LN.
// LA (weight rows a whole number of 128-byte lines from a line-aligned base):
// each chunk row is fetched as the whole lines that hold it, starting at the
// line of its first byte, so no load instruction touches part of a line (up to
// a line more per row than the chunk's bytes; the lines a neighbouring
// wavefront also fetches are cache hits). The staged chunk row then begins
// (chunk byte offset mod 128) bytes into the staged lines. Same arithmetic.
// split: this workgroup's K split.
template <class F, int M, int NW, int CH, bool BF, int MODE, int RPW, bool NT, bool LN, bool LA>
__device__ __forceinline__ void gemv_stream_body(const void *__restrict__ a,
                                                 const uint8_t *__restrict__ w,
                                                 float *__restrict__ y, int N, int K, int ks,
                                                 int split)
{
    using C = GemvStreamCfg<F, M, NW, CH, BF, RPW, LA>;
    using R = GemvRows<BF, M>;
    constexpr bool AL = MODE == 1, PA = MODE == 2;
    static_assert(!AL || C::AH == 1, "A operands read from LDS need the whole chunk's in one pass");
    static_assert(!PA || !BF, "prepared operands are made from f32 activations");
    static_assert(!LN || MODE != 1, "row-group loops keep the A operands in registers");
    constexpr int NACC = R::NACC;
    constexpr uint32_t ES = BF ? 2 : 4;           // bytes per activation
    constexpr int ASTRIDE = 4 * C::NI * 16;       // A bytes per block

    // Per wavefront: [staged weight bytes | A operands].
    // PA needs no A area: its operands go straight to registers.
    constexpr int kLdsPerWave = PA ? C::WBYTES : C::LDS_PER_WAVE;
    __shared__ __attribute__((aligned(16))) uint8_t s_mem[NW * kLdsPerWave];
    __shared__ float s_part[LN ? 2 : 1][NW][M][16];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int j = lane & 15, g = lane >> 4;
    int n0 = blockIdx.x * RPW;
    const int nblk = K >> 5;
    const uint32_t row_bytes = (uint32_t)nblk * F::kBytes;
    uint8_t *s_w = s_mem + wave * kLdsPerWave;
    uint8_t *s_a = s_w + C::WBYTES;

    // The workgroup's K split: blocks [kb_lo, kb_hi) (the whole row unless the
    // call splits K across workgroups, blockIdx.y being the split; each split
    // then writes its own partial y, M x N f32, at y + split M N), a whole
    // number of CH-block chunks (the host picks CH so). The chunks are dealt
    // to the wavefronts in turn: wavefront w takes chunks w, w + NW, ... So
    // the chunk size depends only on K, not on how K divides among the
    // wavefronts, and long rows keep 16-block chunks (more bytes in flight).
    const int kb_lo = split * ks, kb_hi = min(kb_lo + ks, nblk);
    const int wb0 = kb_lo + wave * C::CH;       // this wavefront's first chunk
    constexpr int kStride = NW * C::CH;         // ... and the step to its next
    y += (size_t)split * (size_t)M * (size_t)N;

    // Loader role (GemvStreamCfg): in load i < RH NG, row lrow + 8 (i % RH),
    // column lcol + 8 (i / RH); in the tail load, row trow, column
    // 8 NG + tcol (clamped to the last column: surplus lanes re-read it).
    // Each load thus touches one cache line's worth per row, eight rows.
    const int lrow = lane >> 3, lcol = lane & 7, trow = lane / C::TLPR, tcol = lane % C::TLPR;
    uint32_t row_off0, row_off1, tail_off;
    auto set_rows = [&](int r0) __attribute__((always_inline)) {
        row_off0 = (uint32_t)min(r0 + lrow, N - 1) * row_bytes;
        row_off1 = (uint32_t)min(r0 + lrow + 8, N - 1) * row_bytes;
        tail_off = (uint32_t)min(r0 + trow, N - 1) * row_bytes +
                   16u * (uint32_t)(8 * C::NG + min(tcol, C::TC > 0 ? C::TC - 1 : 0));
    };
    set_rows(n0);

    u32x4 wreg[C::NLOAD];
    // Four activations per half group: f32, or bfloat16 pairs.
    using AV = std::conditional_t<BF, uint2, float4>;
    AV areg[C::EPL][2];
    // Entry r of a lane: A pass h = r / EPP, group c = sq + QN (r % EPP) of
    // that pass (block h CHH + c / 4 of the chunk, lane group gg = c % 4), row
    // sm: elements lo(gg)..lo(gg)+3 and hi(gg)..hi(gg)+3. Activations are
    // requested first (vmcnt drains in issue order), so their split overlaps
    // the weight loads.
    const int sq = lane % C::QN, sm = lane / C::QN;
    const int sm_ld = min(sm, M - 1);
    const uint8_t *a8 = reinterpret_cast<const uint8_t *>(a);
    // Every lane issues every load (surplus lanes re-read an in-bounds group or
    // column that is then ignored), so the compiler's in-order wait counts are
    // exact and the first half of a chunk waits only for its own loads.
    auto fetch_impl = [&](int cb0, auto acts_c) __attribute__((always_inline)) {
        constexpr bool kActs = decltype(acts_c)::value && !PA;
#pragma unroll
        for (int r = 0; r < (kActs ? C::EPL : 0); ++r) {
            const int c = min(sq + C::QN * (r % C::EPP), 4 * C::CHH - 1);
            const int b = (r / C::EPP) * C::CHH + (c >> 2), gg = c & 3;
            const uint32_t off = ((uint32_t)sm_ld * K + (uint32_t)(cb0 + b) * 32 + F::a_lo(1) * gg) * ES;
            areg[r][0] = *reinterpret_cast<const AV *>(a8 + off);
            areg[r][1] = *reinterpret_cast<const AV *>(a8 + off + ES * (F::a_hi(0) - F::a_lo(0)));
        }
        // The scheduling barriers keep the loads in column order. LA: the
        // columns count from the line that holds the chunk's first byte.
        const uint32_t cbo = ((uint32_t)cb0 * F::kBytes) & (LA ? ~127u : ~0u);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < C::RH * C::NG; ++i) {
            const u32x4 *src = reinterpret_cast<const u32x4 *>(
                w + ((i % C::RH ? row_off1 : row_off0) + cbo + 16u * (uint32_t)(lcol + 8 * (i / C::RH))));
            wreg[i] = NT ? __builtin_nontemporal_load(src) : *src;
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (C::TC > 0)
        {
            const u32x4 *src = reinterpret_cast<const u32x4 *>(w + (tail_off + cbo));
            wreg[C::RH * C::NG] = NT ? __builtin_nontemporal_load(src) : *src;
        }
        // Issue point: the weight pointer escapes into an empty asm statement
        // with a memory clobber, so no pass sinks the loads below this line,
        // and the scheduling barrier keeps later work (which waits on loads)
        // from being hoisted above them.
        asm volatile("" ::"s"(w) : "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    auto fetch = [&](int cb0) __attribute__((always_inline)) { fetch_impl(cb0, std::true_type{}); };
    auto fetch_w = [&](int cb0) __attribute__((always_inline)) { fetch_impl(cb0, std::false_type{}); };

    // Unconditional, so no copies of the loaded registers are needed after a
    // branch (they would wait for the loads). A wavefront without blocks
    // (possible only when the workgroup's share is short) fetches the last full
    // chunk of the row, K/32 >= CH, and never reads it.
    // A operands of a chunk live in registers (set by split_activations, or
    // for PA loaded by fetch_ops).
    f16x8 aop[C::CH];
    // PA: the chunk's prepared operands, operand (b, g, i) of block cb0 + b at
    // ((cb0 + b) * 4 + g) * NI + i. Only lanes j < NI load: the other A rows
    // belong to no activation row and only fill MFMA rows that are never read.
    const u32x4 *ops = static_cast<const u32x4 *>(a);
    auto fetch_ops = [&](int cb0) __attribute__((always_inline)) {
        if constexpr (PA) {
            if (j < C::NI) {
#pragma unroll
                for (int b = 0; b < C::CH; ++b)
                    aop[b] = bitcast<f16x8>(ops[((size_t)(cb0 + b) * 4 + g) * C::NI + j]);
            }
        }
    };
    // The first chunk: prepared operands first (their loads drain before the
    // weights', so part 0 waits only for its own weight bytes), then weights.
    fetch_ops(min(wb0, nblk - C::CH));
    fetch(min(wb0, nblk - C::CH));
    // Clamped, so the address stays inside the A area even where the read is
    // masked off.
    // Operand reads: lane (g, j) reads A row j of lane group g; the swizzle
    // depends on the block's parity (ASTRIDE is a whole number of slots).
    const int jr = min(j, C::NI - 1);
    const uint8_t *a_lane0 = s_a + (g * C::NI + (jr ^ a_swz<C::NI>(0, g))) * 16;
    const uint8_t *a_lane1 = s_a + (g * C::NI + (jr ^ a_swz<C::NI>(1, g))) * 16;
    // The decode's exponent pattern in a VGPR (one v_mov at kernel start; no
    // MFMA is in flight there).
    const uint32_t magic_v = magic_vgpr<F>();

    float ysum[R::NOUT];
#pragma unroll
    for (int h = 0; h < R::NOUT; ++h)
        ysum[h] = 0.0f;

    // Activation split of the chunk whose loads are in areg: per-row scale
    // from the chunk's own max |a|, then the two-term A operands into s_a.
    // It runs as soon as those loads land, never across a loop back edge, so
    // no copy of the loaded registers is kept alive while the weight loads are
    // being issued.
    int pexp[M];
    if constexpr (PA) {
        // The per-row exponents follow the operands.
        const int *row_exp = reinterpret_cast<const int *>(ops + (size_t)nblk * 4 * C::NI);
#pragma unroll
        for (int m = 0; m < M; ++m)
            pexp[m] = row_exp[m];
    }
    auto split_activations = [&]() __attribute__((always_inline)) {
        if constexpr (PA)
            return;
        // Every entry of a lane belongs to its row sm: one running maximum,
        // then one reduction over the lanes of the row. Clamped entries repeat
        // a group of the same row and lanes sm >= M a row that is never used,
        // so neither needs a mask here.
        // f32: |a| through v_max3_f32 with absolute-value modifiers, two
        // elements an instruction; bfloat16: the halves compared as integers
        // (non-negative floats order like their bit patterns), two at a time.
        uint32_t mb = 0;
        u16x2 mb16 = {0, 0};
        float mf = 0.0f;
        constexpr uint32_t kAbs2 = 0x7fff7fffu;
#pragma unroll
        for (int r = 0; r < C::EPL; ++r) {
            if constexpr (BF) {
                const uint2 L = areg[r][0], H = areg[r][1];
                mb16 = __builtin_elementwise_max(
                    mb16, __builtin_elementwise_max(bitcast<u16x2>(L.x & kAbs2), bitcast<u16x2>(L.y & kAbs2)));
                mb16 = __builtin_elementwise_max(
                    mb16, __builtin_elementwise_max(bitcast<u16x2>(H.x & kAbs2), bitcast<u16x2>(H.y & kAbs2)));
            } else {
                const float4 L = areg[r][0], H = areg[r][1];
                mf = max3_abs(max3_abs(mf, L.x, L.y), L.z, L.w);
                mf = max3_abs(max3_abs(mf, H.x, H.y), H.z, H.w);
            }
        }
        if constexpr (BF)
            mb = (uint32_t)max(mb16.x, mb16.y) << 16;
        else
            mb = __float_as_uint(mf);
        const float am = lane_run_max_nonneg<C::QN>(__uint_as_float(mb));
        const int pe = BF ? row_scale_exp_bf16<F>(am) : row_scale_exp<F>(am);
        // Lane m QN holds row m's exponent; the epilogue needs every row's.
#pragma unroll
        for (int m = 0; m < M; ++m)
            pexp[m] = __builtin_amdgcn_readlane(pe, m * C::QN);
        // Each pass writes the groups of its blocks and reads them back as A
        // operands at once; the next pass reuses the same LDS area. A lane's
        // groups share its lane group gg = sq % 4 and block parity (sq / 4) % 2
        // (QN / 4 is even), so its slots within a block are fixed.
        const int gg = sq & 3, sw = a_swz<C::NI>(sq >> 2, gg);
        const int slot_hi = gg * C::NI + ((BF ? sm : 2 * sm) ^ sw);
        const int slot_lo = gg * C::NI + ((2 * sm + 1) ^ sw);
#pragma unroll
        for (int h = 0; h < C::AH; ++h) {
        if (h > 0)
            wave_lds_sync();   // the previous pass's reads precede these writes
#pragma unroll
        for (int rr = 0; rr < C::EPP; ++rr) {
            const int r = h * C::EPP + rr, c = sq + C::QN * rr;
            if ((C::QN * C::EPP == 4 * C::CHH || c < 4 * C::CHH) && (C::MP == M || sm < M)) {
                uint8_t *blk = s_a + (c >> 2) * ASTRIDE;
                if constexpr (BF) {
                    const uint2 L = areg[r][0], H = areg[r][1];
                    const int pl = pe + F::kHiLog2;
                    const float v[8] = {ldexpf(bf16_lo(L.x), pl), ldexpf(bf16_lo(L.y), pl),
                                        ldexpf(bf16_hi(L.x), pl), ldexpf(bf16_hi(L.y), pl),
                                        ldexpf(bf16_lo(H.x), pe), ldexpf(bf16_lo(H.y), pe),
                                        ldexpf(bf16_hi(H.x), pe), ldexpf(bf16_hi(H.y), pe)};
                    f16x8 hi;
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        hi[s] = (f16)v[s];
                    *reinterpret_cast<u32x4 *>(blk + slot_hi * 16) = bitcast<u32x4>(hi);
                } else {
                    // sc the power of two (times 2^kHiLog2 on slots 0..3);
                    // slots (L.x, L.z, L.y, L.w, H.x, H.z, H.y, H.w).
                    const float sh = ldexpf(1.0f, pe), sl = (float)(1 << F::kHiLog2) * sh;
                    const float4 L = areg[r][0], H = areg[r][1];
                    uint32_t h0, h1, h2, h3, l0, l1, l2, l3;
                    split2_pair(L.x, L.z, sl, h0, l0);
                    split2_pair(L.y, L.w, sl, h1, l1);
                    split2_pair(H.x, H.z, sh, h2, l2);
                    split2_pair(H.y, H.w, sh, h3, l3);
                    *reinterpret_cast<u32x4 *>(blk + slot_hi * 16) = u32x4{h0, h1, h2, h3};
                    *reinterpret_cast<u32x4 *>(blk + slot_lo * 16) = u32x4{l0, l1, l2, l3};
                }
            }
        }
        // A operands into registers now, while the weight bytes are still in
        // flight. Only lanes j < NI read: the other A rows belong to no
        // activation row and only fill MFMA output rows that are never read.
        wave_lds_sync();
        if (!AL && j < C::NI) {
#pragma unroll
            for (int b = h * C::CHH; b < (h + 1) * C::CHH; ++b)
                aop[b] = *reinterpret_cast<const f16x8 *>((b & 1 ? a_lane1 : a_lane0) +
                                                          (b - h * C::CHH) * ASTRIDE);
        }
        }
    };
    const f32x4 zero4 = {0.f, 0.f, 0.f, 0.f};
    split_activations();
    // Epilogue of one row group: wavefront partials into LDS (buffer buf),
    // then summed in wavefront order and stored.
    auto write_out = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < R::NOUT; ++h) {
            const int m = R::row(g, h);
            if (m < M && j < RPW)
                s_part[buf][wave][m][j] = ysum[h];
            ysum[h] = 0.0f;
        }
        __syncthreads();
        if (tid < M * RPW) {
            const int m = tid / RPW, jj = tid % RPW, n = n0 + jj;
            float sum = 0.0f;
#pragma unroll
            for (int ww = 0; ww < NW; ++ww)
                sum += s_part[buf][ww][m][jj];
            if (n < N)
                y[(size_t)m * N + n] = sum;
        }
    };
    // LN: this workgroup's row group (it walks groups blockIdx.x, + gridDim.x, ...).
    int rg = blockIdx.x, it = 0;
    for (int cb0 = wb0; cb0 < kb_hi; cb0 += LN ? 0 : kStride) {
        const bool more = LN ? (rg + (int)gridDim.x) * RPW < N : cb0 + kStride < kb_hi;
        // The chunk is contracted in NPART parts. Part p needs only loads
        // [0, loads_for(end of p)) of every lane, which drain first (vmcnt
        // counts in issue order), so its decode and MFMAs run while the rest of
        // the chunk is still arriving.
        auto stage = [&](auto i0_c, auto i1_c) __attribute__((always_inline)) {
            constexpr int I0 = decltype(i0_c)::value, I1 = decltype(i1_c)::value;
#pragma unroll
            for (int i = I0; i < I1; ++i) {
                if (i < C::RH * C::NG)
                    *reinterpret_cast<u32x4 *>(s_w + (lrow + 8 * (i % C::RH)) * C::RS +
                                               16 * (lcol + 8 * (i / C::RH))) = wreg[i];
                else if (tcol < C::TC)
                    *reinterpret_cast<u32x4 *>(s_w + trow * C::RS + 16 * (8 * C::NG + tcol)) = wreg[i];
            }
        };
        float acc[NACC];
#pragma unroll
        for (int r = 0; r < NACC; ++r)
            acc[r] = 0.0f;
        // Block b of the staged row starts at byte kBytes b; read_qs realigns the
        // quant bytes of lane group g where they straddle dwords. All MFMAs of a
        // part are issued before its scale FMAs, so the matrix-core latency
        // overlaps the decode of the following blocks.
        // Lane j decodes weight row j; with eight rows per workgroup the
        // upper eight MFMA columns repeat row 7 and are never read.
        // LA: the chunk starts (cb0 kBytes) mod 128 bytes into the staged lines.
        const uint8_t *wl = s_w + min(j, C::RPW - 1) * C::RS +
                            (LA ? (((uint32_t)cb0 * F::kBytes) & 127u) : 0u);
        const uint32_t *wrow32 = reinterpret_cast<const uint32_t *>(wl);
        auto contract = [&](auto b0_c, auto b1_c) __attribute__((always_inline)) {
            constexpr int B0 = decltype(b0_c)::value, B1 = decltype(b1_c)::value;
            f32x4 Cv[B1 - B0];
            float d[B1 - B0];
            static_for<B0, B1>([&](auto b_c) __attribute__((always_inline)) {
                constexpr int b = decltype(b_c)::value;
                uint32_t x[F::kQsDwords];
                read_qs<F, b>(wrow32, g, x);
                d[b - B0] = f16_bits_to_f32(*reinterpret_cast<const uint16_t *>(wl + b * F::kBytes));
                f16x8 av;
                if constexpr (AL)
                    av = *reinterpret_cast<const f16x8 *>((b & 1 ? a_lane1 : a_lane0) + b * ASTRIDE);
                else
                    av = aop[b];
                Cv[b - B0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(av, F::decode(x, magic_v),
                                                                     zero4, 0, 0, 0);
            });
#pragma unroll
            for (int u = 0; u < B1 - B0; ++u)
#pragma unroll
                for (int r = 0; r < NACC; ++r)
                    acc[r] = fmaf(d[u], Cv[u][r], acc[r]);
            // Keep every MFMA result register allocated up to here: rows this
            // lane does not accumulate would otherwise be handed to the next
            // decode while the MFMA is still writing them (a stall on each).
#pragma unroll
            for (int u = 0; u < B1 - B0; ++u)
                asm volatile("" ::"v"(Cv[u]));
        };
        // Undo this chunk's scale (and the factor 2^kHiLog2) on its partial.
        auto finish_chunk = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int h = 0; h < R::NOUT; ++h) {
                const int m = R::row(g, h);
                int pm = 0;
#pragma unroll
                for (int mm = 0; mm < M; ++mm)
                    if (mm == m)
                        pm = pexp[mm];
                ysum[h] += ldexpf(BF ? acc[h] : acc[2 * h] + acc[2 * h + 1], -pm - F::kHiLog2);
            }
        };
        // In the row-group loops, and where a wavefront walks several chunks
        // (the launches with the A operands in LDS or plain loads), a group's
        // or chunk's bytes have mostly landed by the time its wavefront gets
        // to them (they were requested one round earlier), so parts no longer
        // overlap arrival and only chain LDS round trips: Q4_0 takes 8-block
        // parts there (1 x 14336 x 4096 8.75 -> 8.48 us, 1 x 11008 x 2048
        // 5.19 -> 4.98, 1 x 4096 x 14336 8.51 -> 8.25, bfloat16 1 x 4096 x
        // 14336 8.37 -> 7.86; Q8_0 was 1-2% slower with fewer parts). With
        // whole-line loads a Q4_0 chunk's first and second halves wait for the
        // same loads as the parts within them, so they are one part each there
        // too (1 x 4096 x 4096 4.15 -> 4.11 us, 4 x 4096 x 4096 5.22 -> 5.12).
        constexpr bool kRounds = LN || (MODE == 1 && RPW == 16) || (MODE == 0 && !NT);
        constexpr int NPX = ((kRounds || LA) && F::kBytes == kQ4Bytes) ? CH / 8 : C::NPART;
        for_each_part<NPX>([&](auto p_c) __attribute__((always_inline)) {
            constexpr int P = decltype(p_c)::value;
            constexpr int B0 = P * C::CH / NPX, B1 = (P + 1) * C::CH / NPX;
            constexpr int L0 = C::loads_for(B0), L1 = C::loads_for(B1);
            stage(std::integral_constant<int, L0>{}, std::integral_constant<int, L1>{});
            auto run_part = [&]() __attribute__((always_inline)) {
                wave_lds_sync();
                contract(std::integral_constant<int, B0>{}, std::integral_constant<int, B1>{});
            };
            if constexpr (P < NPX - 1) {
                run_part();
            } else if (LN && more) {
                // Every load of this group is staged: prefetch the next
                // group's weights for the same chunk, then finish this one.
                set_rows((rg + (int)gridDim.x) * RPW);
                fetch_w(cb0);
                run_part();
                finish_chunk();
            } else if (more) {
                // Every load of this chunk is staged: prefetch the next chunk,
                // finish this one, then split the next chunk's activations (PA:
                // load its prepared operands, once this chunk's are used). The
                // fetch and the split sit in one branch, so the loaded
                // activation registers never meet a join.
                fetch(cb0 + kStride);
                run_part();
                finish_chunk();
                wave_lds_sync();   // this chunk's LDS reads precede the next chunk's writes
                split_activations();
                fetch_ops(cb0 + kStride);
            } else {
                run_part();
                finish_chunk();
            }
        });
        if constexpr (LN) {
            write_out(it & 1);
            if (!more)
                break;
            rg += (int)gridDim.x;
            ++it;
            n0 = rg * RPW;
            wave_lds_sync();   // this group's LDS reads precede the next group's writes
        }
    }
    if constexpr (!LN)
        write_out(0);
}

template <class F, int M, int NW, int CH, bool BF, int MODE, int RPW = 16, bool NT = false,
          bool LN = false, bool LA = false>
__global__ __launch_bounds__(64 * NW) void k_gemv_stream(const void *__restrict__ a,
                                                        const uint8_t *__restrict__ w,
                                                        float *__restrict__ y, int N, int K,
                                                        int ks)
{
    gemv_stream_body<F, M, NW, CH, BF, MODE, RPW, NT, LN, LA>(a, w, y, N, K, ks, (int)blockIdx.y);
}

// True where every weight row is a whole number of 128-byte lines from a
// line-aligned base (K % 2048 == 0 in either format), so the streaming kernels
// can fetch whole lines (LA). Against loads that start at each chunk's first
// byte (same process, cold, bit-identical results): 1 x 4096 x 4096 4.24 ->
// 4.15 us, 2 x 4096 x 4096 4.85 -> 4.60, 1 x 4096 x 2048 3.44 -> 3.28, Q8_0
// 1 x 4096 x 4096 5.64 -> 5.31. With them the non-temporal hint pays on every
// launch (it cost 1.5-5% with partial lines where a compute unit holds two
// workgroups or a wavefront walks several chunks): 1 x 14336 x 4096 9.07 ->
// 8.69 us, 1 x 4096 x 14336 8.86 -> 8.56, 1 x 11008 x 2048 5.66 -> 5.16, Q8_0
// 1 x 4096 x 14336 13.7 -> 12.5.
template <class F>
inline bool gemv_rows_line_aligned(const uint8_t *w, int K)
{
    return ((size_t)(K / 32) * F::kBytes) % 128 == 0 && ((uintptr_t)w & 127u) == 0;
}

}  // namespace q4k
