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
#include "f64.h"
#include "launch.h"
#include "validate.h"

namespace q4k {

constexpr int kRouteThreads = 1024, kRouteWaves = kRouteThreads / 64;
constexpr int kMaxExperts = Q4_MAX_EXPERTS, kMaxTopK = Q4_MAX_TOP_K;
static_assert(kMaxExperts == kRouteThreads, "one thread per expert in the scans");

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

// W: keys of a wavefront's token in expert order, where groups are ranked.
template <int W = 1>
struct RouteLds {
    int cursor[kMaxExperts];                          // next position of each expert
    int part[kRouteWaves];
    union {
        uint16_t waves[kRouteWaves][kMaxExperts];     // slots of a batch, by wavefront and expert
        double vals[kRouteWaves][W];                  // not needed any more when slots are placed
    };
};

// Exclusive prefix sum over the workgroup's threads.
__device__ __forceinline__ int exclusive_scan(int v, int *part)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int s = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int u = __shfl_up(s, d);
        if (lane >= d)
            s += u;
    }
    if (lane == 63)
        part[wave] = s;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < wave; ++w)
        before += part[w];
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
    for (int b = 0; b < n; b += kRouteThreads) {
        const int used = (min(n - b, kRouteThreads) + 63) / 64;   // wavefronts with slots
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

using q4v::route_chunk;
using q4v::route_chunks;
constexpr int kOneChunk = q4v::kRouteOneChunk;

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
        __builtin_amdgcn_wave_barrier();
        for (int u = 0; u < n; ++u)
            if ((tid & 63) < top_k)
                atomicAdd(&l.cursor[to(u)[tid & 63]], 1);
    }
    __syncthreads();
    const int count = tid < E ? l.cursor[tid] : 0;
    if (counts) {
        if (tid < E)
            counts[(size_t)blockIdx.x * E + tid] = count;
        return;
    }
    const int at = exclusive_scan(count, l.part);
    if (tid < E)
        offsets[tid] = at;
    if (tid == 0)
        offsets[E] = T * top_k;
    place(l, [&](int i) { return (int)s_ids[i]; }, 0, T * top_k, E, bits, at, order);
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
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = min((int)(threadIdx.x & 63) + 64 * i, E - 1);
        x.bias[i] = g.bias ? g.bias[e] : 0.0f;
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
            __builtin_amdgcn_wave_barrier();
            const uint64_t kept = best_groups(vals, g, E, lanes);
            __builtin_amdgcn_wave_barrier();
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

// Chunk c's slots to their places: thread (p, e) sums expert e's counts over
// the chunks c' = p mod parts, all of them and those before c.
__global__ __launch_bounds__(kRouteThreads) void k_route_place(const int *__restrict__ ids,
                                                              const int *__restrict__ counts,
                                                              int *__restrict__ offsets,
                                                              int *__restrict__ order, int T, int E,
                                                              int top_k, int chunk, int chunks,
                                                              int bits)
{
    __shared__ RouteLds<> l;
    __shared__ int sums[2][kRouteThreads];
    const int tid = threadIdx.x, c = blockIdx.x;
    const int width = 1 << bits, parts = kRouteThreads / width;   // E <= width <= 1024
    const int e = tid & (width - 1), p = tid >> bits;
    int all = 0, before = 0;
    if (e < E) {
#pragma unroll 8
        for (int k = p; k < chunks; k += parts) {
            const int v = counts[(size_t)k * E + e];
            all += v;
            before += k < c ? v : 0;
        }
    }
    sums[0][tid] = all;
    sums[1][tid] = before;
    __syncthreads();
    all = before = 0;
    if (tid < E) {
        for (int q = 0; q < parts; ++q) {
            all += sums[0][(q << bits) + tid];
            before += sums[1][(q << bits) + tid];
        }
    }
    const int first = exclusive_scan(all, l.part);
    if (c == 0) {
        if (tid < E)
            offsets[tid] = first;
        if (tid == 0)
            offsets[E] = T * top_k;
    }
    const int s0 = c * chunk * top_k, n = (min((c + 1) * chunk, T) - c * chunk) * top_k;
    place(l, [&](int i) { return ids[s0 + i]; }, s0, n, E, bits, first + before, order);
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
    return launch_kernel(k_route_place, dim3((unsigned)chunks), dim3(kRouteThreads), 0, st, ids, counts,
                         offsets, order, T, E, top_k, chunk, chunks, expert_bits(E));
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

hipError_t launch_route_groups(const float *logits, const RouteGroups &g, int *ids, float *weights,
                               int *offsets, int *order, void *workspace, int T, int E, int top_k,
                               hipStream_t st)
{
    const int chunk = route_chunk(T), chunks = route_chunks(T);
    int *counts = chunks > 1 ? static_cast<int *>(workspace) : nullptr;
    int lanes = 6;
    while (g.n_groups << lanes > 64)
        --lanes;
    auto kernel = g.top_groups < g.n_groups ? groups_kernel<true>(E) : groups_kernel<false>(E);
    hipError_t e = launch_kernel(kernel, dim3((unsigned)chunks), dim3(kRouteThreads), 0, st, logits, g,
                                 lanes, ids, weights, offsets, order, counts, T, E, top_k, chunk,
                                 expert_bits(E));
    if (e != hipSuccess || !counts)
        return e;
    return launch_place(ids, counts, offsets, order, T, E, top_k, st);
}

}  // namespace q4k
