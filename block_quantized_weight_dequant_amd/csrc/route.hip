// The router of a mixture of experts: for each token the top_k largest of E
// logits (the lowest expert among equal ones) and their softmax weights, and
// the slots (t, j) = t top_k + j sorted by expert, which the grouped products
// read.
//
// Bound by latency: 8192 tokens of 64 experts are 2 MB. One wavefront takes a
// token, its lanes the experts; a step of the selection is a maximum over the
// wavefront (DPP), a ballot for the lowest expert that has it, and one key
// cleared. Logits compare as unsigned keys (sign-flipped bit patterns, -0 as
// +0), so the choice is exact and needs no float compare of NaN; a cleared key
// is 0 and every other at least 1, so top_k <= E distinct experts always come
// out, whatever the logits hold.
//
// The sort is a counting sort that keeps equal experts in slot order without
// atomics that could change it: workgroup c counts its tokens' experts
// (counts are sums, their order does not matter), the second launch adds up
// the counts of all chunks and of the earlier ones, and 64 slots at a time get
// their rank from ballots over the bits of the expert (lanes with the same
// expert, those before mine). Up to 64 tokens one workgroup does all of
// it in one launch.
//
// With scores, a bias and groups (q4_route_groups) the keys are f64, s + bias, and
// so are the groups' sums: scores that differ in f32's last place would come out
// in either order, and two f64 roundings almost never. s takes some 25 f64
// operations an expert. A step of the selection then compares the keys' upper
// halves, and the lower ones only where several experts share the largest.
#include <algorithm>

#include "f64.h"
#include "launch.h"
#include "validate.h"

namespace q4k {

constexpr int kRouteThreads = 1024, kRouteWaves = kRouteThreads / 64;
constexpr int kMaxExperts = Q4_MAX_EXPERTS, kMaxTopK = Q4_MAX_TOP_K;

// Order LDS traffic between the lanes of one wavefront: its LDS operations
// execute in issue order, so it is enough that the compiler keeps them there.
__device__ __forceinline__ void wave_lds_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        v += __shfl_xor(v, d);
    return v;
}

// Order-preserving key of a logit, at least 1.
__device__ __forceinline__ uint32_t logit_key(float v)
{
    const uint32_t u = __float_as_uint(v + 0.0f);
    return max((u >> 31) ? ~u : (u | 0x80000000u), 1u);
}

__device__ __forceinline__ float key_logit(uint32_t k)
{
    return __uint_as_float((k >> 31) ? (k & 0x7FFFFFFFu) : ~k);
}

// Tokens t and t + kRouteWaves by one wavefront, side by side (their steps are
// chains of short latencies): lane l holds experts l, l + 64, ... of each. Lane
// j < top_k ends with choice j. s_ids(i) takes token i's choices.
template <int V, class Ids>
__device__ __forceinline__ void route_tokens(const float *__restrict__ logits, int E, int top_k,
                                             int renorm, int *__restrict__ ids,
                                             float *__restrict__ weights, const int (&tok)[2],
                                             int n, Ids s_ids)
{
    const int lane = threadIdx.x & 63;
    uint32_t key[2][V], first[2][V], my_key[2] = {0, 0}, top[2] = {0, 0};
    int my_id[2] = {0, 0};
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const float *x = logits + (size_t)tok[u] * (size_t)E;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 64 * i;
            const float v = x[min(e, E - 1)];
            key[u][i] = first[u][i] = e < E ? logit_key(v) : 0u;
        }
    }
    for (int j = 0; j < top_k; ++j) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t m = key[u][0];
#pragma unroll
            for (int i = 1; i < V; ++i)
                m = max(m, key[u][i]);
            const uint32_t best = wave_max_u32(m);
            // The lowest expert with the best key: the first i in which any lane
            // has it, and there the lowest lane.
            int id = -1;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const uint64_t has = __ballot(key[u][i] == best);
                if (id < 0 && has) {
                    const int l = __builtin_ctzll(has);
                    id = 64 * i + l;
                    key[u][i] = lane == l ? 0u : key[u][i];
                }
            }
            if (j == 0)
                top[u] = best;
            if (lane == j)
                my_key[u] = best, my_id[u] = id;
        }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        // exp(l - max) is in [0, 1]; a row of -inf (every expert masked) weighs 0.
        const float mx = key_logit(top[u]);
        const bool none = mx == -__builtin_inff();
        const float w = lane < top_k && !none ? expf(key_logit(my_key[u]) - mx) : 0.0f;
        float s = w;
        if (!renorm) {
            s = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (first[u][i] != 0u && !none)
                    s += expf(key_logit(first[u][i]) - mx);
        }
        const float total = wave_sum(s);
        if (u < n && lane < top_k) {
            const size_t at = (size_t)tok[u] * (size_t)top_k + lane;
            ids[at] = my_id[u];
            weights[at] = none ? 0.0f : w / total;
            s_ids(u)[lane] = (uint16_t)my_id[u];
        }
    }
}

// NT threads, at most MAX_E experts; W: 8-byte keys of a wavefront's token in
// expert order, where it needs them.
template <int W = 1, int NT = kRouteThreads, int MAX_E = kMaxExperts>
struct RouteLds {
    static constexpr int kThreads = NT;
    static_assert(MAX_E <= NT, "one thread per expert in the scans");
    int cursor[MAX_E];                              // next position of each expert
    int part[NT / 64];
    union {
        uint16_t waves[NT / 64][MAX_E];             // slots of a batch, by wavefront and expert
        double vals[NT / 64][W];                    // not needed any more when slots are placed
        uint64_t keys[NT / 64][W];
    };
};

// Inclusive prefix sum over the wavefront: DPP within rows of 16, then each row's
// last lane into the next row, and lane 31 into the upper half.
template <int CTRL, int ROWS>
__device__ __forceinline__ int add_from(int v)
{
    return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int wave_scan(int v)
{
    v = add_from<0x111, 0xF>(v);   // row_shr 1
    v = add_from<0x112, 0xF>(v);   // row_shr 2
    v = add_from<0x114, 0xF>(v);   // row_shr 4
    v = add_from<0x118, 0xF>(v);   // row_shr 8
    v = add_from<0x142, 0xA>(v);   // row_bcast 15 into rows 1 and 3
    return add_from<0x143, 0xC>(v);   // row_bcast 31 into rows 2 and 3
}

// Exclusive prefix sum over the workgroup's NW wavefronts.
template <int NW>
__device__ __forceinline__ int exclusive_scan(int v, int (&part)[NW])
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int s = wave_scan(v);
    if (lane == 63)
        part[wave] = s;
    __syncthreads();
    int before = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w)
        before += w < wave ? part[w] : 0;
    __syncthreads();
    return before + s - v;
}

// Place slots s0 .. s0 + n - 1, whose experts expert(0) .. expert(n - 1) are
// (below E; bits: of an expert number). Thread e < E passes the first position
// of its expert in `at`.
template <class Lds, class Fn>
__device__ __forceinline__ void place(Lds &l, Fn expert, int s0, int n, int E, int bits, int at,
                                      int *__restrict__ order)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int b = 0; b < n; b += Lds::kThreads) {
        const int used = (min(n - b, Lds::kThreads) + 63) / 64;   // wavefronts with slots
        if (tid < E)
            for (int w = 0; w < used; ++w)
                l.waves[w][tid] = 0;
        __syncthreads();
        const int i = b + tid;
        const bool in = i < n;
        const int e = in ? expert(i) : 0;
        uint64_t same = __ballot(in);
        for (int bit = 0; bit < bits; ++bit) {
            const uint64_t set = __ballot((e >> bit) & 1);
            same &= (e >> bit) & 1 ? set : ~set;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        if (in && rank == 0)
            l.waves[wave][e] = (uint16_t)__popcll(same);
        __syncthreads();
        if (tid < E) {      // counts -> slots of the batch before each wavefront's
            int before = 0;
#pragma unroll 4
            for (int w = 0; w < used; ++w) {
                const int c = l.waves[w][tid];
                l.waves[w][tid] = (uint16_t)before;
                before += c;
            }
            l.cursor[tid] = at;
            at += before;
        }
        __syncthreads();
        if (in)
            order[l.cursor[e] + l.waves[wave][e] + rank] = s0 + i;
        __syncthreads();
    }
}

// The counts of a chunk: 16 bits each where they fit (and their padded rows fit the
// workspace), in rows of whole 16 bytes, so that the second launch, in which every
// workgroup adds up the whole table, reads half the bytes in wide loads.
__host__ __device__ inline bool route_narrow(int E, int chunk, int top_k) { return E >= 8 && chunk <= 65535 / top_k; }
__host__ __device__ inline size_t route_pitch(int E) { return ((size_t)E + 7) / 8 * 8; }

using q4v::route_chunk;
using q4v::route_chunks;
constexpr int kOneChunk = q4v::kRouteOneChunk;

// What follows when the chunk's experts are counted in l.cursor: the counts, or,
// where one workgroup does all of it, the sort.
template <class Lds>
__device__ __forceinline__ void route_sort(Lds &l, const uint16_t *s_ids, int *__restrict__ offsets,
                                           int *__restrict__ order, int *__restrict__ counts, int T, int E,
                                           int top_k, int chunk, int bits)
{
    const int tid = threadIdx.x;
    __syncthreads();
    const int count = tid < E ? l.cursor[tid] : 0;
    if (counts) {
        if (route_narrow(E, chunk, top_k)) {
            if (tid < (int)route_pitch(E))
                reinterpret_cast<uint16_t *>(counts)[(size_t)blockIdx.x * route_pitch(E) + tid] = (uint16_t)count;
        } else if (tid < E) {
            counts[(size_t)blockIdx.x * E + tid] = count;
        }
        return;
    }
    const int at = exclusive_scan(count, l.part);
    if (tid < E)
        offsets[tid] = at;
    if (tid == 0)
        offsets[E] = T * top_k;
    place(l, [&](int i) { return (int)s_ids[i]; }, 0, T * top_k, E, bits, at, order);
}

// One workgroup's chunk: tokens(tok, n, to) chooses the experts of n tokens (the
// second tok repeats another if n is 1) and leaves the choices of the u-th at
// to(u). counts: [chunks][E], or null when one workgroup does all of it.
template <class Lds, class Tokens>
__device__ __forceinline__ void route_workgroup(Lds &l, uint16_t *s_ids, Tokens tokens,
                                                int *__restrict__ offsets, int *__restrict__ order,
                                                int *__restrict__ counts, int T, int E, int top_k,
                                                int chunk, int bits)
{
    const int tid = threadIdx.x, wave = tid >> 6;
    if (tid < E)
        l.cursor[tid] = 0;
    __syncthreads();
    const int t0 = blockIdx.x * chunk, t1 = min(t0 + chunk, T);
    for (int t = t0 + wave; t < t1; t += 2 * kRouteWaves) {
        const int tok[2] = {t, min(t + kRouteWaves, t1 - 1)}, n = t + kRouteWaves < t1 ? 2 : 1;
        // One workgroup alone keeps every token's choice, in slot order.
        auto to = [&](int u) __attribute__((always_inline)) {
            return s_ids + (counts ? (wave * 2 + u) * kMaxTopK : (tok[u] - t0) * top_k);
        };
        tokens(tok, n, to);
        wave_lds_sync();
        for (int u = 0; u < n; ++u)
            if ((tid & 63) < top_k)
                atomicAdd(&l.cursor[to(u)[tid & 63]], 1);
    }
    route_sort(l, s_ids, offsets, order, counts, T, E, top_k, chunk, bits);
}

template <int V>
__global__ __launch_bounds__(kRouteThreads) void k_route(const float *__restrict__ logits,
                                                        int *__restrict__ ids,
                                                        float *__restrict__ weights,
                                                        int *__restrict__ offsets,
                                                        int *__restrict__ order,
                                                        int *__restrict__ counts, int T, int E,
                                                        int top_k, int renorm, int chunk, int bits)
{
    __shared__ RouteLds<> l;
    __shared__ uint16_t s_ids[kOneChunk * kMaxTopK];   // at least two tokens a wavefront
    const auto tokens = [&](const int (&tok)[2], int n, auto to) __attribute__((always_inline)) {
        route_tokens<V>(logits, E, top_k, renorm, ids, weights, tok, n, to);
    };
    route_workgroup(l, s_ids, tokens, offsets, order, counts, T, E, top_k, chunk, bits);
}

// An expert's place in the order of choice: larger first. 0 takes no part, 1 (a
// masked expert) comes last; f64 keys, in two halves, are larger.
struct Key {
    uint32_t hi, lo;
};
__device__ __forceinline__ Key f64_key(double v)
{
    const u32x2 b = bitcast<u32x2>(v + 0.0);   // -0 as +0
    const uint32_t flip = (uint32_t)((int)b.y >> 31);
    return {b.y ^ (flip | 0x80000000u), b.x ^ flip};
}

__device__ const float kNoBias = 0.0f;

// What a wavefront keeps of its V experts lane + 64 i for all its tokens.
template <int V>
struct Experts {
    float bias[V];
    int bit[V];   // the first lane of the expert's group
};

// 2^lanes lanes rank a group's experts: as many as n_groups leave of the 64.
template <int V, bool GROUPED>
__device__ __forceinline__ Experts<V> load_experts(const RouteGroups &g, int E, int lanes)
{
    Experts<V> x;
    const int size = E / g.n_groups;
    const float *bias = g.bias ? g.bias : &kNoBias;   // loads that need no branch stay in flight together
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = min((int)(threadIdx.x & 63) + 64 * i, E - 1);
        x.bias[i] = bias[g.bias ? e : 0];
        x.bit[i] = GROUPED ? (e / size) << lanes : 0;
    }
    return x;
}

// The groups of one token that can be chosen: bits at their first lanes. vals:
// the wavefront's E keys in expert order, masked ones -inf.
__device__ __forceinline__ uint64_t best_groups(const double *vals, const RouteGroups &g, int E, int lanes)
{
    const int lane = threadIdx.x & 63, size = E / g.n_groups, mine = lane >> lanes, step = 1 << lanes;
    const double none = -__builtin_inf();
    double first = none, second = none;
    if (mine < g.n_groups)
        for (int k = lane & (step - 1); k < size; k += step) {
            const double v = vals[mine * size + k];
            second = fmax(second, fmin(first, v));
            first = fmax(first, v);
        }
    for (int d = 1; d < step; d <<= 1) {
        const double f = __shfl_xor(first, d), s = __shfl_xor(second, d);
        second = fmax(fmin(first, f), fmax(second, s));
        first = fmax(first, f);
    }
    const double score = g.group_best == 2 ? first + second : first;
    int rank = 0;
    for (int j = 0; j < g.n_groups; ++j) {
        const double other = readlane_f64(score, j << lanes);
        rank += other > score || (other == score && j < mine);
    }
    return __ballot(mine < g.n_groups && rank < g.top_groups);
}

// Tokens tok[0 .. U - 1] by one wavefront; lane j < top_k ends with choice j.
template <int V, int U, bool GROUPED, class Ids>
__device__ __forceinline__ void choose_tokens(const float *__restrict__ logits, const RouteGroups &g,
                                              const Experts<V> &x, double *vals, int lanes, int E,
                                              int top_k, int *__restrict__ ids,
                                              float *__restrict__ weights, const int *tok, int n, Ids s_ids)
{
    const int lane = threadIdx.x & 63;
    const float ninf = -__builtin_inff();
    float v[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < V; ++i)
            v[u][i] = logits[(size_t)tok[u] * (size_t)E + min(lane + 64 * i, E - 1)];

    double s[U][V], my_s[U];
    Key key[U][V];
    int my_id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        bool there[V];   // an expert, and not masked (NaN masks)
#pragma unroll
        for (int i = 0; i < V; ++i)
            there[i] = lane + 64 * i < E && v[u][i] > ninf;
        if (g.sigmoid) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const double z = fmin(fmax((double)v[u][i], -700.0), 700.0);
                s[u][i] = there[i] ? rcp_f64(1.0 + exp_f64(-z)) : 0.0;
            }
        } else {
            uint32_t m = logit_key(ninf);
#pragma unroll
            for (int i = 0; i < V; ++i)
                m = max(m, there[i] ? logit_key(v[u][i]) : 0u);
            const double mx = (double)key_logit(wave_max_u32(m));
            double sum = 0.0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const double e = exp_f64(fmax((double)v[u][i] - mx, -700.0));
                s[u][i] = there[i] ? e : 0.0;
                sum += s[u][i];
            }
            const double r = rcp_f64(fmax(wave_sum_f64(sum), 0x1p-1000));
#pragma unroll
            for (int i = 0; i < V; ++i)
                s[u][i] *= r;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const double k = s[u][i] + (double)x.bias[i];
            there[i] = there[i] && x.bias[i] > ninf;
            key[u][i] = there[i] ? f64_key(k) : Key{0u, lane + 64 * i < E ? 1u : 0u};
            if (GROUPED && lane + 64 * i < E)
                vals[lane + 64 * i] = there[i] ? k : -__builtin_inf();
        }
        if constexpr (GROUPED) {
            wave_lds_sync();
            const uint64_t kept = best_groups(vals, g, E, lanes);
            wave_lds_sync();
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (!(kept >> x.bit[i] & 1))
                    key[u][i] = {0u, 0u};
        }
        my_id[u] = 0;
        my_s[u] = 0.0;
    }

    for (int j = 0; j < top_k; ++j) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            uint32_t m = key[u][0].hi;
#pragma unroll
            for (int i = 1; i < V; ++i)
                m = max(m, key[u][i].hi);
            const uint32_t best = wave_max_u32(m);
            uint64_t has[V];
            int many = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                has[i] = __ballot(key[u][i].hi == best);
                many += __popcll(has[i]);
            }
            if (many > 1) {
                m = 0;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    m = max(m, key[u][i].hi == best ? key[u][i].lo : 0u);
                const uint32_t low = wave_max_u32(m);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    has[i] = __ballot(key[u][i].hi == best && key[u][i].lo == low);
            }
            // The lowest expert: the first i in which any lane has it, and there the lowest lane.
            int id = -1;
            double sel = 0.0;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (id < 0 && has[i]) {
                    const int l = __builtin_ctzll(has[i]);
                    id = 64 * i + l;
                    sel = readlane_f64(s[u][i], l);
                    if (lane == l)
                        key[u][i] = {0u, 0u};
                }
            if (lane == j) {
                my_id[u] = id;
                my_s[u] = best ? sel : 0.0;   // 0: masked
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const double total = wave_sum_f64(my_s[u]);
        const double w = g.renorm ? (total > 0.0 ? my_s[u] * rcp_f64(total) : 0.0) : my_s[u];
        if (u < n && lane < top_k) {
            const size_t at = (size_t)tok[u] * (size_t)top_k + lane;
            ids[at] = my_id[u];
            weights[at] = (float)(w * (double)g.scale);
            s_ids(u)[lane] = (uint16_t)my_id[u];
        }
    }
}

// How four tokens share a wavefront, 16 lanes (a DPP row) each: 2^lanes lanes
// hold a group's experts, `per` neighbours each; without a choice of groups the
// row is one group.
struct RouteRows {
    int groups, lanes, size, per;
};

// Largest, and sum, over the 16 lanes of a row, in every one of them.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ float dpp_of(float v) { return __uint_as_float(dpp_u32<CTRL>(__float_as_uint(v))); }
template <int CTRL>
__device__ __forceinline__ double dpp_of(double v) { return dpp_f64<CTRL>(v); }
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return fmax(a, b); }
__device__ __forceinline__ float smaller(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ double smaller(double a, double b) { return fmin(a, b); }
// The middle one of a >= b and c.
__device__ __forceinline__ float middle(float a, float b, float c) { return __builtin_amdgcn_fmed3f(a, b, c); }
__device__ __forceinline__ double middle(double a, double b, double c) { return fmax(b, fmin(a, c)); }
template <class K>
__device__ __forceinline__ K row_max(K v)
{
    v = larger(v, dpp_of<0xB1>(v));
    v = larger(v, dpp_of<0x4E>(v));
    v = larger(v, dpp_of<0x141>(v));
    return larger(v, dpp_of<0x140>(v));
}
__device__ __forceinline__ uint32_t row_max(uint32_t v)
{
    v = max(v, dpp_u32<0xB1>(v));
    v = max(v, dpp_u32<0x4E>(v));
    v = max(v, dpp_u32<0x141>(v));
    return max(v, dpp_u32<0x140>(v));
}
__device__ __forceinline__ double row_sum(double v)
{
    v += dpp_f64<0xB1>(v);
    v += dpp_f64<0x4E>(v);
    v += dpp_f64<0x141>(v);
    return v + dpp_f64<0x140>(v);
}

// Falling order, by Batcher's merge exchange (63 exchanges of 16, 191 of 32).
template <int N>
__device__ __forceinline__ void sort_falling(uint32_t (&v)[N])
{
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const uint32_t a = v[i + j], b = v[i + j + k];
                        v[i + j] = max(a, b);
                        v[i + j + k] = min(a, b);
                    }
}

// The value itself, which the compiler then computes where it stands: sunk under the
// condition of a later choice, each score would be a chain of dependent operations by
// itself instead of one among many.
template <class K>
__device__ __forceinline__ K at_once(K v)
{
    asm volatile("" : "+v"(v));
    return v;
}

// Score of one logit that is not masked. Softmax: top is the row's largest logit,
// share the reciprocal of its sum.
template <bool SIGMOID>
__device__ __forceinline__ double score_of(float v, double top, double share)
{
    if constexpr (SIGMOID)
        return rcp_f64(1.0 + exp_f64(fmin(fmax(-(double)v, -700.0), 700.0)));
    else
        return exp_f64(fmax((double)v - top, -700.0)) * share;
}

// A lane's experts e0 .. e0 + n - 1 and what they share for all tokens: `unit`
// steps of a key's code to 1, and keys whose codes are up to `blur` steps apart may
// come in either order.
template <int CAP, class K>
struct RowExperts {
    float bias[CAP];   // of places without an expert: -inf
    int e0, n, group;
    K unit, margin;    // groups' sums up to `margin` apart may be in either order
    uint32_t blur;
};
// A code's low bits: the lane (4) and the place in it.
template <int CAP>
constexpr int kPlaceBits = CAP <= 16 ? 4 : 5;
template <int CAP>
constexpr int kTagBits = 4 + kPlaceBits<CAP>;
template <int CAP>
constexpr uint32_t kMostSteps = (1u << (32 - kTagBits<CAP>)) - 1024;
constexpr uint32_t kMaskedCode = 1;

// CAP floats from byte `at` on, zeros past the buffer: whole 16-byte loads at any
// 4-byte alignment, without a branch, so that all stay in flight together.
template <int CAP>
__device__ __forceinline__ void load_row(float (&v)[CAP], __amdgpu_buffer_rsrc_t b, uint32_t at)
{
#pragma unroll
    for (int i = 0; i < CAP; i += 4) {
        const u32x4 q = __builtin_amdgcn_raw_buffer_load_b128(b, at + 4 * i, 0, 0);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            v[i + k] = __uint_as_float(q[k]);
    }
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_buffer(const float *p, size_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<float *>(p), 0, (int)(bytes < 0x7FFFFFFF ? bytes : 0x7FFFFFFF), 0x00020000);
}

template <int CAP, class K>
__device__ __forceinline__ void place_row_experts(RowExperts<CAP, K> &x, const float *logits, const RouteGroups &g,
                                                  const RouteRows &r, int E)
{
    const int p = threadIdx.x & 15, part = p & ((1 << r.lanes) - 1);
    x.group = p >> r.lanes;
    x.n = x.group < r.groups ? min(max(r.size - part * r.per, 0), r.per) : 0;
    x.e0 = x.n ? x.group * r.size + part * r.per : 0;
    load_row(x.bias, row_buffer(g.bias ? g.bias : logits, g.bias ? (size_t)E * 4 : 0), (uint32_t)x.e0 * 4);
}

// Scores lie in [0, 1], so keys span at most R = 1 more than the finite biases and 0
// (hi + lo). Errors of a key: f64 (softmax): far below a step, which two roundings
// to steps can turn into two. f32 (sigmoid), with u = 2^-24 and B the largest |bias|:
// the exponent's rounding moves the score by s (1 - s) |l| 2^-23.7 <= 0.3 u, the
// exponential by s (1 - s) 2 u <= 0.5 u, 1 + e and the reciprocal by s 3 u: 3.8 u;
// the sum with the bias by (1 + B) u; the distance from the largest key and its
// product with `unit` by R u each. So two keys whose codes are in the wrong order are
// less than (10 + 2 B + 4 R) u apart in them, 16 steps at most, and one step more by
// the roundings of both to steps.
template <int CAP, class K>
__device__ __forceinline__ void scale_row_experts(RowExperts<CAP, K> &x)
{
    float hi = 0.0f, lo = 0.0f;
#pragma unroll
    for (int i = 0; i < CAP; ++i) {
        const float b = fabsf(x.bias[i]) < __builtin_inff() ? x.bias[i] : 0.0f;   // 0 of NaN too
        hi = larger(hi, b);   // places past the lane's experts only widen the range
        lo = smaller(lo, b);
        x.bias[i] = i < x.n ? x.bias[i] : -__builtin_inff();
    }
    hi = row_max(hi);
    lo = row_max(-lo);
    const float range = 1.0f + (hi + lo), unit = (float)kMostSteps<CAP> * 0.999999f * __builtin_amdgcn_rcpf(range);
    x.unit = (K)unit;
    if constexpr (sizeof(K) == 4) {
        const float most = larger(hi, lo), err = 0x1p-24f * (10.0f + 2.0f * most + 4.0f * range);
        // Four keys' errors, and the roundings of two sums and of the comparison.
        x.margin = 0x1p-20f + 12 * 0x1p-24f * (1.0f + most);
        // Where the biases' range leaves f32 all is uncertain (the masked code is 1000 away).
        x.blur = err * unit < 500.0f ? (uint32_t)(err * unit) + 2u : ~0u;
    } else {
        x.margin = 0x1p-48 * (double)range;
        x.blur = 2u;
    }
}

// LDS of a wavefront of rows: the tokens' logits by lane and place (a lane's at a
// pitch that spreads them over the banks), and the keys of a token that is chosen
// exactly.
constexpr int kRowThreads = 512, kRowWaves = kRowThreads / 64, kRowTopK = 15;
template <int CAP>
constexpr int kRowExperts = CAP <= 16 ? 256 : 512;
template <int CAP>
struct RowLds {
    static constexpr int kPitch = kRowExperts<CAP> / 16 + 1;
    float logits[64 * kPitch];
    union {
        double vals[kRowExperts<CAP>];
        uint64_t keys[kRowExperts<CAP>];
    };
};

// One token by the whole wavefront, with keys in f64: into l.vals, masked ones
// -inf; returns the groups that can be chosen (bits as best_groups').
template <bool GROUPED, bool SIGMOID, class Lds>
__device__ __forceinline__ uint64_t exact_keys(const float *__restrict__ row, const RouteGroups &g, int lanes,
                                               Lds &l, int E)
{
    const int lane = threadIdx.x & 63;
    const float ninf = -__builtin_inff();
    double top = 0.0, share = 1.0;
    if constexpr (!SIGMOID) {
        uint32_t m = logit_key(ninf);
        for (int e = lane; e < E; e += 64)
            m = max(m, row[e] > ninf ? logit_key(row[e]) : 0u);
        const float t = key_logit(wave_max_u32(m));
        top = t > ninf ? (double)t : 0.0;
        double sum = 0.0;
        for (int e = lane; e < E; e += 64)
            sum += row[e] > ninf ? score_of<SIGMOID>(row[e], top, 1.0) : 0.0;
        share = rcp_f64(fmax(wave_sum_f64(sum), 0x1p-1000));
    }
    const float *bias = g.bias ? g.bias : row;
    wave_lds_sync();
#pragma unroll 4
    for (int e = lane; e < E; e += 64) {
        const float v = row[e], b = g.bias ? bias[e] : 0.0f;
        l.vals[e] = (v > ninf) & (b > ninf) ? score_of<SIGMOID>(v, top, share) + (double)b : -__builtin_inf();
    }
    wave_lds_sync();
    return GROUPED ? best_groups(l.vals, g, E, lanes) : 0;
}

// One token's choices by the whole wavefront, the lowest expert among equals.
// Small and slow: hardly a token needs it.
template <bool GROUPED, bool SIGMOID, class Lds>
__device__ __forceinline__ void choose_exactly(const float *__restrict__ row, const RouteGroups &g, int lanes,
                                               Lds &l, int E, int top_k, uint16_t *out)
{
    const int lane = threadIdx.x & 63, size = E / g.n_groups;
    const uint64_t kept = exact_keys<GROUPED, SIGMOID>(row, g, lanes, l, E);
    wave_lds_sync();
    for (int e = lane; e < E; e += 64) {
        const double v = l.vals[e];
        const Key k = f64_key(v);
        const uint64_t key = v > -__builtin_inf() ? (uint64_t)k.hi << 32 | k.lo : 1u;
        l.keys[e] = !GROUPED || (kept >> (e / size << lanes) & 1) ? key : 0u;
    }
    for (int j = 0; j < top_k; ++j) {
        wave_lds_sync();
        uint64_t mine = 0;
        int at = lane;
        for (int e = lane; e < E; e += 64)
            if (l.keys[e] > mine)
                mine = l.keys[e], at = e;
        const uint32_t hi = wave_max_u32((uint32_t)(mine >> 32));
        const uint32_t lo = wave_max_u32((uint32_t)(mine >> 32) == hi ? (uint32_t)mine : 0u);
        const bool best = mine == ((uint64_t)hi << 32 | lo);
        const int id = 2 * kMaxExperts - (int)wave_max_u32(best ? (uint32_t)(2 * kMaxExperts - at) : 0u);
        wave_lds_sync();
        if (lane == 0) {
            out[j] = (uint16_t)id;
            l.keys[id] = 0;
        }
    }
    wave_lds_sync();
}

// Tokens by four rows of a wavefront: tok is uniform within a row, v its logits,
// `in` where it is not a repetition. Choice j goes to out[j], and with its weight to
// ids and weights.
//
// A key (s + bias: sigmoid scores in f32 here, softmax scores in f64) becomes a
// code of 24 bits (23 with 17 to 32 experts a lane), its distance from the row's
// largest in steps of the range that keys can have, with the expert's lane and its
// place in the lane in the bits below, so that equal codes are in the order of their experts. A lane sorts its
// codes once, and a step of the selection is a maximum over the row's heads (four DPP
// moves) for four tokens at a time, and one head taken off. Codes near enough to be
// in the wrong order are taken along, and ordered by f64 keys, which the weights need
// of each candidate anyway. Where that does not settle it (more than 16 candidates)
// the token is chosen again, exactly: so are all tokens whose scores agree in f32,
// as saturated ones without a bias do (logits all above 14 or below -14: 32 tokens 8 of
// 256 45.5 us for 8.6, 8192 tokens 52.8 for 15.7).
template <int CAP, bool GROUPED, bool SIGMOID, class K>
__device__ __forceinline__ void choose_rows(float (&v)[CAP], const float *__restrict__ logits, const RouteGroups &g,
                                            const RouteRows &r, const RowExperts<CAP, K> &x, RowLds<CAP> &l, int lanes,
                                            int E, int top_k, int *__restrict__ ids, float *__restrict__ weights,
                                            int tok, bool in, uint16_t *out)
{
    const int lane = threadIdx.x & 63, p = lane & 15;
    const float ninf = -__builtin_inff();
    const K none = -(K)__builtin_inf();
#pragma unroll
    for (int i = 0; i < CAP; ++i)
        l.logits[lane * l.kPitch + i] = v[i];
    double top = 0.0, share = 1.0;
    K key[CAP];
    if constexpr (SIGMOID) {
#pragma unroll
        for (int i = 0; i < CAP; ++i)
            key[i] = at_once(__builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v[i] * -1.44269504f)) + x.bias[i]);
    } else {
        float m = ninf;
#pragma unroll
        for (int i = 0; i < CAP; ++i)
            m = fmaxf(m, i < x.n ? v[i] : ninf);   // of NaN the other
        m = row_max(m);
        top = m > ninf ? (double)m : 0.0;
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < CAP; ++i) {
            key[i] = at_once(score_of<SIGMOID>(v[i], top, 1.0));
            sum += (i < x.n) & (v[i] > ninf) ? key[i] : 0.0;
        }
        share = rcp_f64(fmax(row_sum(sum), 0x1p-1000));
#pragma unroll
        for (int i = 0; i < CAP; ++i)
            key[i] = key[i] * share + (double)x.bias[i];
    }
    K first = none, second = none;
#pragma unroll
    for (int i = 0; i < CAP; ++i) {
        // Masked by the logit (-inf or NaN) or the bias, or absent. (The minimum of
        // NaN and a number is NaN here.)
        key[i] = __builtin_elementwise_minimum(v[i], x.bias[i]) > ninf ? key[i] : none;
        if (GROUPED)
            second = middle(first, second, key[i]);
        first = larger(first, key[i]);
    }
    bool open = x.n > 0;   // the lane's experts can be chosen
    const K mine = first;
    if constexpr (GROUPED) {
        const auto merge = [&](K f, K s) __attribute__((always_inline)) {
            second = larger(smaller(first, f), larger(second, s));
            first = larger(first, f);
        };
        if (r.lanes > 0)
            merge(dpp_of<0xB1>(first), dpp_of<0xB1>(second));
        if (r.lanes > 1)
            merge(dpp_of<0x4E>(first), dpp_of<0x4E>(second));
        if (r.lanes > 2)
            merge(dpp_of<0x141>(first), dpp_of<0x141>(second));
        const K score = g.group_best == 2 ? first + second : first;
        // Lanes of the row (whole groups, by turning it) whose sum is better for
        // certain, and those that may be, the lane's own group among them.
        int ahead = 0, maybe = 1;
        const K above = score + x.margin, below = score - x.margin;
        unroll<15>([&](auto turn) __attribute__((always_inline)) {
            const K other = dpp_of<0x121 + turn.value>(score);   // row_ror 1 .. 15
            ahead += other > above;
            maybe += !(other < below);
        });
        ahead >>= r.lanes;
        maybe >>= r.lanes;
        const bool sure = (maybe <= g.top_groups) | (ahead >= g.top_groups);
        open = open & (maybe <= g.top_groups);
        // Sums too near to tell, once in some ten thousand tokens: by f64 keys.
        uint64_t unsure = __ballot((x.n > 0) & !sure);
        while (unsure) {
            const int u = __builtin_ctzll(unsure) & 48;
            unsure &= ~(0xFFFFull << u);
            const size_t t = (size_t)__builtin_amdgcn_readlane(tok, u);
            const uint64_t kept = exact_keys<GROUPED, SIGMOID>(logits + t * (size_t)E, g, lanes, l, E);
            if ((lane & 48) == u)
                open = (x.n > 0) & (kept >> (x.group << lanes) & 1) != 0;
        }
    }
    const K most = row_max(open ? mine : none);
    constexpr int PLACE = kPlaceBits<CAP>, PLACES = (1 << PLACE) - 1, TAG = kTagBits<CAP>;
    uint32_t code[CAP];
#pragma unroll
    for (int i = 0; i < CAP; ++i) {
        const K far = smaller(larger((most - key[i]) * x.unit, (K)0), (K)kMostSteps<CAP>);
        const uint32_t steps = key[i] > none ? (1u << (32 - TAG)) - 1u - (uint32_t)far : kMaskedCode;
        code[i] = open & (i < x.n) ? steps << TAG | (uint32_t)((15 - p) << PLACE | (PLACES - i)) : 0u;
    }
    sort_falling(code);
    // Codes are taken until what is left is certain to be smaller than the top_k-th. A
    // lane offers its eight largest: a row that would take more of one is not certain.
    constexpr int LIST = CAP < 8 ? CAP : 8;
    uint32_t taken = 0, best = 0;   // lane j's: the j-th code
    int offered = 0;
    const auto take = [&](int j) __attribute__((always_inline)) {
        taken = p == j ? best : taken;
        if (code[0] == best) {
            ++offered;
#pragma unroll
            for (int i = 0; i + 1 < LIST; ++i)
                code[i] = code[i + 1];
            code[LIST - 1] = 0;
        }
    };
#pragma unroll 1
    for (int j = 0; j < top_k; ++j) {
        best = row_max(code[0]);
        take(j);
    }
    const uint32_t last = best;
    bool more = true;
#pragma unroll 1
    for (int j = top_k; j < 16; ++j) {
        best = row_max(code[0]);
        more = ((last >> TAG) - (best >> TAG) <= x.blur) & (best >> TAG > kMaskedCode);
        if (!__ballot(more))
            break;
        take(j);
    }
    const bool doubt = more | ((CAP > LIST) & (offered >= LIST) & (x.n > LIST));

    // Lane p: candidate p, its score in f64.
    wave_lds_sync();
    const int from = (lane & 48) + 15 - (int)(taken >> PLACE & 15u), at = PLACES - (int)(taken & (uint32_t)PLACES);
    int id = __shfl(x.e0, from) + at;
    float logit = l.logits[from * l.kPitch + (at < CAP ? at : 0)];
    bool masked = taken >> TAG <= kMaskedCode;
    double s = at_once(score_of<SIGMOID>(logit, top, share));
    s = masked ? 0.0 : s;
    const uint32_t next = dpp_u32<0x101>(taken);   // row_shl 1: the lane after
    const bool near = (next >> TAG > kMaskedCode) & ((taken >> TAG) - (next >> TAG) <= x.blur);
    if (__ballot(near)) {
        // Some neighbours may be in the wrong order: by their f64 keys, then, the lowest
        // expert among equals.
        const float b = (g.bias ? g.bias : logits)[masked ? 0 : id];
        const double k = masked ? -__builtin_inf() : s + (double)(g.bias ? b : 0.0f);
        int rank = 0;
        unroll<15>([&](auto turn) __attribute__((always_inline)) {
            constexpr int C = 0x121 + turn.value;
            const double other = dpp_of<C>(k);
            rank += (other > k) | ((other == k) & ((int)dpp_u32<C>((uint32_t)(masked ? 4096 + p : id)) < (masked ? 4096 + p : id)));
        });
        const int to = ((lane & 48) + rank) * 4;   // a permutation of the row
        id = __builtin_amdgcn_ds_permute(to, id);
        const u32x2 h = bitcast<u32x2>(s);
        s = bitcast<double>((u32x2){(uint32_t)__builtin_amdgcn_ds_permute(to, (int)h.x), (uint32_t)__builtin_amdgcn_ds_permute(to, (int)h.y)});
    }
    if (p < top_k)
        out[p] = (uint16_t)id;
    uint64_t unsure = __ballot(doubt);
    while (unsure) {
        const int u = __builtin_ctzll(unsure) & 48;
        unsure &= ~(0xFFFFull << u);
        wave_lds_sync();
        const int t = __builtin_amdgcn_readlane(tok, u);
        const uint64_t o = reinterpret_cast<uint64_t>(out);
        uint16_t *to = reinterpret_cast<uint16_t *>((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(o >> 32), u) << 32 |
                                                    (uint32_t)__builtin_amdgcn_readlane((int)o, u));
        choose_exactly<GROUPED, SIGMOID>(logits + (size_t)t * (size_t)E, g, lanes, l, E, top_k, to);
        if ((lane & 48) == u && p < top_k) {
            id = out[p];
            logit = logits[(size_t)tok * (size_t)E + id];
            s = at_once(score_of<SIGMOID>(logit, top, share));
            s = (logit > ninf) & ((g.bias ? g.bias[id] : 0.0f) > ninf) ? s : 0.0;
        }
    }

    s = p < top_k ? s : 0.0;
    const double total = row_sum(s);
    const double w = g.renorm ? (total > 0.0 ? s * rcp_f64(total) : 0.0) : s;
    if (in && p < top_k) {
        const size_t to = (size_t)tok * (size_t)top_k + p;
        ids[to] = id;
        weights[to] = (float)(w * (double)g.scale);
    }
}

// Up to 512 experts in rows of lanes, CAP or fewer a lane, four tokens a wavefront at
// a time: 32 / 2048 / 8192 tokens of 512 experts in 8 groups 12.9 / 19.9 / 22.7 us
// (48.3 / 55.5 / 79.6 with a wavefront a token); 32 / 8192 of 256 8.6 / 15.7.
template <int CAP, bool GROUPED, bool SIGMOID>
__global__ __launch_bounds__(kRowThreads) void k_route_rows(const float *__restrict__ logits, RouteGroups g,
                                                           RouteRows r, int lanes, int *__restrict__ ids,
                                                           float *__restrict__ weights, int *__restrict__ offsets,
                                                           int *__restrict__ order, int *__restrict__ counts, int T,
                                                           int E, int top_k, int chunk, int bits)
{
    using K = std::conditional_t<SIGMOID, float, double>;
    __shared__ RouteLds<1, kRowThreads, kRowExperts<CAP>> l;
    __shared__ RowLds<CAP> rows[kRowWaves];
    __shared__ uint16_t s_ids[kOneChunk * kRowTopK];   // the choices of a chunk that is alone, or of a pass
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int t0 = blockIdx.x * chunk, t1 = min(t0 + chunk, T);
    // The chunk's logits span less than 2^31 bytes: 256 of them all are on the card.
    const __amdgpu_buffer_rsrc_t all = row_buffer(logits + (size_t)t0 * (size_t)E, (size_t)(T - t0) * (size_t)E * 4);
    RowExperts<CAP, K> x;
    float v[CAP];
    place_row_experts(x, logits, g, r, E);
    const auto fetch = [&](int t) __attribute__((always_inline)) {
        load_row(v, all, ((uint32_t)min(t + (lane >> 4), t1 - 1) - (uint32_t)t0) * (uint32_t)E * 4u + (uint32_t)x.e0 * 4u);
    };
    fetch(t0 + 4 * wave);
    if (tid < E)
        l.cursor[tid] = 0;
    __syncthreads();
    scale_row_experts(x);
    for (int t = t0 + 4 * wave; t < t1; t += 4 * kRowWaves) {
        const int mine = t + (lane >> 4), tok = min(mine, t1 - 1);
        uint16_t *out = s_ids + (mine - t0) % kOneChunk * top_k;
        choose_rows<CAP, GROUPED, SIGMOID>(v, logits, g, r, x, rows[wave], lanes, E, top_k, ids, weights, tok, mine < t1, out);
        if (t + 4 * kRowWaves < t1)
            fetch(t + 4 * kRowWaves);
        if (mine < t1 && (lane & 15) < top_k)
            atomicAdd(&l.cursor[out[lane & 15]], 1);
        wave_lds_sync();
    }
    route_sort(l, s_ids, offsets, order, counts, T, E, top_k, chunk, bits);
}

// Every size: one token a wavefront at a time. 16 experts a lane (above 256) spill 41
// (GROUPED: 84) registers: 32 / 8192 tokens 8 of 1024 in 8 groups 54 / 93 us.
template <int V, bool GROUPED>
__global__ __launch_bounds__(kRouteThreads) void k_route_groups(const float *__restrict__ logits,
                                                               RouteGroups g, int lanes,
                                                               int *__restrict__ ids,
                                                               float *__restrict__ weights,
                                                               int *__restrict__ offsets,
                                                               int *__restrict__ order,
                                                               int *__restrict__ counts, int T,
                                                               int E, int top_k, int chunk, int bits)
{
    constexpr int U = V <= 4 ? 2 : 1;   // two tokens' keys and scores of 16 experts a lane do not fit the registers
    __shared__ RouteLds<GROUPED ? 64 * V : 1> l;
    __shared__ uint16_t s_ids[kOneChunk * kMaxTopK];
    const Experts<V> x = load_experts<V, GROUPED>(g, E, lanes);
    double *vals = l.vals[GROUPED ? threadIdx.x >> 6 : 0];
    const auto tokens = [&](const int (&tok)[2], int n, auto to) __attribute__((always_inline)) {
        if constexpr (U == 2) {
            choose_tokens<V, 2, GROUPED>(logits, g, x, vals, lanes, E, top_k, ids, weights, tok, n, to);
        } else {
            for (int u = 0; u < n; ++u)
                choose_tokens<V, 1, GROUPED>(logits, g, x, vals, lanes, E, top_k, ids, weights, tok + u, 1,
                                             [&](int) __attribute__((always_inline)) { return to(u); });
        }
    };
    route_workgroup(l, s_ids, tokens, offsets, order, counts, T, E, top_k, chunk, bits);
}

// The slots of chunks c0 = blockIdx.x run .. c0 + run - 1 to their places, after the
// sums of the experts' counts over all chunks and over those before c0. NARROW:
// 16-bit counts, eight experts a thread.
template <bool NARROW>
__global__ __launch_bounds__(kRouteThreads) void k_route_place(const int *__restrict__ ids,
                                                              const int *__restrict__ counts,
                                                              int *__restrict__ offsets,
                                                              int *__restrict__ order, int T, int E,
                                                              int top_k, int chunk, int chunks, int run,
                                                              int bits)
{
    constexpr int W = NARROW ? 8 : 1;   // experts a thread
    __shared__ RouteLds<> l;
    __shared__ __align__(16) int sums[2][W * kRouteThreads];
    const int tid = threadIdx.x, c0 = blockIdx.x * run;
    const int s0 = c0 * chunk * top_k, n = ((int)min((long long)(c0 + run) * chunk, (long long)T) - c0 * chunk) * top_k;
    const int mine = ids[s0 + min(tid, n - 1)];   // the first batch's, on its way meanwhile
    // Threads a row of the table, and rows at a time: few, since their sums are added
    // up below one after another.
    const int width = max(1, (1 << bits) / W);
    const int parts = min(min(kRouteThreads / width, chunks > 128 ? 32 : 16), chunks);
    const int q = tid % width, p = tid / width;
    int all[W] = {}, before[W] = {};
    const auto add_rows = [&](auto in_flight) __attribute__((always_inline)) {
        constexpr int N = in_flight.value;
        for (int k0 = p; k0 < chunks; k0 += N * parts) {
            std::conditional_t<NARROW, u32x4, int> v[N];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const size_t k = (size_t)min(k0 + j * parts, chunks - 1);
                if constexpr (NARROW)
                    v[j] = *reinterpret_cast<const u32x4 *>(reinterpret_cast<const uint16_t *>(counts) + k * route_pitch(E) + q * 8);
                else
                    v[j] = counts[k * (size_t)E + q];
            }
            asm volatile("" ::: "memory");   // all of them before the first is used
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int k = k0 + j * parts;
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    int c;
                    if constexpr (NARROW)
                        c = (int)(i & 1 ? v[j][i / 2] >> 16 : v[j][i / 2] & 0xFFFFu);
                    else
                        c = v[j];
                    all[i] += k < chunks ? c : 0;
                    before[i] += k < c0 ? c : 0;   // c0 < chunks
                }
            }
        }
    };
    if (q * W < E && p < parts) {
        if (chunks > 2 * parts)
            add_rows(std::integral_constant<int, 8>{});
        else
            add_rows(std::integral_constant<int, 2>{});
    }
    // Part p's sums at p's row of `width` W experts.
    if constexpr (NARROW) {
#pragma unroll
        for (int i = 0; i < W; i += 4) {
            reinterpret_cast<i32x4 *>(sums[0])[(tid * W + i) / 4] = (i32x4){all[i], all[i + 1], all[i + 2], all[i + 3]};
            reinterpret_cast<i32x4 *>(sums[1])[(tid * W + i) / 4] = (i32x4){before[i], before[i + 1], before[i + 2], before[i + 3]};
        }
    } else {
        sums[0][tid] = all[0];
        sums[1][tid] = before[0];
    }
    __syncthreads();
    int total = 0, ahead = 0;
    if (tid < E)
#pragma unroll 8
        for (int k = 0; k < parts; ++k) {
            total += sums[0][k * width * W + tid];
            ahead += sums[1][k * width * W + tid];
        }
    const int first = exclusive_scan(total, l.part);
    if (c0 == 0) {
        if (tid < E)
            offsets[tid] = first;
        if (tid == 0)
            offsets[E] = T * top_k;
    }
    place(l, [&](int i) { return i < kRouteThreads ? mine : ids[s0 + i]; }, s0, n, E, bits, first + ahead, order);
}

static int expert_bits(int E)
{
    int bits = 0;
    while ((1 << bits) < E)
        ++bits;
    return bits;
}

// The second launch, where there is more than one chunk.
static hipError_t launch_place(const int *ids, const int *counts, int *offsets, int *order, int T, int E,
                               int top_k, hipStream_t st)
{
    const int chunk = route_chunk(T), chunks = route_chunks(T);
    // As many chunks a workgroup as give every thread a slot.
    const int run = std::max(1, kRouteThreads / (chunk * top_k));
    auto kernel = route_narrow(E, chunk, top_k) ? k_route_place<true> : k_route_place<false>;
    return launch_kernel(kernel, dim3((unsigned)((chunks + run - 1) / run)), dim3(kRouteThreads), 0, st, ids,
                         counts, offsets, order, T, E, top_k, chunk, chunks, run, expert_bits(E));
}

hipError_t launch_route(const float *logits, int *ids, float *weights, int *offsets, int *order,
                        void *workspace, int T, int E, int top_k, bool renorm, hipStream_t st)
{
    const int chunk = route_chunk(T), chunks = route_chunks(T);
    int *counts = chunks > 1 ? static_cast<int *>(workspace) : nullptr;
    auto kernel = E <= 64 ? k_route<1> : E <= 128 ? k_route<2> : E <= 256 ? k_route<4> : k_route<16>;
    hipError_t e = launch_kernel(kernel, dim3((unsigned)chunks), dim3(kRouteThreads), 0, st, logits,
                                 ids, weights, offsets, order, counts, T, E, top_k, renorm ? 1 : 0,
                                 chunk, expert_bits(E));
    if (e != hipSuccess || !counts)
        return e;
    return launch_place(ids, counts, offsets, order, T, E, top_k, st);
}

template <bool GROUPED>
static auto groups_kernel(int E)
{
    return E <= 64 ? k_route_groups<1, GROUPED> : E <= 128 ? k_route_groups<2, GROUPED>
         : E <= 256 ? k_route_groups<4, GROUPED> : k_route_groups<16, GROUPED>;
}

template <bool GROUPED, bool SIGMOID>
static auto rows_kernel(int per)
{
    return per <= 4 ? k_route_rows<4, GROUPED, SIGMOID> : per <= 8 ? k_route_rows<8, GROUPED, SIGMOID>
         : per <= 16 ? k_route_rows<16, GROUPED, SIGMOID> : k_route_rows<32, GROUPED, SIGMOID>;
}

hipError_t launch_route_groups(const float *logits, const RouteGroups &g, int *ids, float *weights,
                               int *offsets, int *order, void *workspace, int T, int E, int top_k,
                               hipStream_t st)
{
    const int chunk = route_chunk(T), chunks = route_chunks(T);
    int *counts = chunks > 1 ? static_cast<int *>(workspace) : nullptr;
    const bool grouped = g.top_groups < g.n_groups;
    int lanes = 6;
    while (g.n_groups << lanes > 64)
        --lanes;
    // Rows of 16 lanes hold up to 16 groups, 32 experts a lane, and 15 choices with the one after them.
    RouteRows r = {grouped ? g.n_groups : 1, 4, 0, 0};
    while (r.groups << r.lanes > 16 && r.lanes > 0)
        --r.lanes;
    r.size = E / r.groups;
    r.per = (r.size + (1 << r.lanes) - 1) >> r.lanes;
    hipError_t e;
    if (r.groups <= 16 && r.per <= 32 && top_k <= kRowTopK) {
        auto kernel = grouped ? (g.sigmoid ? rows_kernel<true, true>(r.per) : rows_kernel<true, false>(r.per))
                              : (g.sigmoid ? rows_kernel<false, true>(r.per) : rows_kernel<false, false>(r.per));
        e = launch_kernel(kernel, dim3((unsigned)chunks), dim3(kRowThreads), 0, st, logits, g, r, lanes, ids, weights,
                          offsets, order, counts, T, E, top_k, chunk, expert_bits(E));
        return e != hipSuccess || !counts ? e : launch_place(ids, counts, offsets, order, T, E, top_k, st);
    }
    auto kernel = grouped ? groups_kernel<true>(E) : groups_kernel<false>(E);
    e = launch_kernel(kernel, dim3((unsigned)chunks), dim3(kRouteThreads), 0, st, logits, g,
                                 lanes, ids, weights, offsets, order, counts, T, E, top_k, chunk,
                                 expert_bits(E));
    if (e != hipSuccess || !counts)
        return e;
    return launch_place(ids, counts, offsets, order, T, E, top_k, st);
}

}  // namespace q4k
