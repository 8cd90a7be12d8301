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
#include "device_common.h"
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

struct RouteLds {
    int cursor[kMaxExperts];                      // next position of each expert
    int part[kRouteWaves];
    uint16_t waves[kRouteWaves][kMaxExperts];     // slots of a batch, by wavefront and expert
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
template <class Fn>
__device__ __forceinline__ void place(RouteLds &l, Fn expert, int s0, int n, int E, int bits, int at,
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

// counts: [chunks][E], or null when one workgroup does all of it.
template <int V>
__global__ __launch_bounds__(kRouteThreads) void k_route(const float *__restrict__ logits,
                                                        int *__restrict__ ids,
                                                        float *__restrict__ weights,
                                                        int *__restrict__ offsets,
                                                        int *__restrict__ order,
                                                        int *__restrict__ counts, int T, int E,
                                                        int top_k, int renorm, int chunk, int bits)
{
    __shared__ RouteLds l;
    __shared__ uint16_t s_ids[kOneChunk * kMaxTopK];   // at least two tokens a wavefront
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
        route_tokens<V>(logits, E, top_k, renorm, ids, weights, tok, n, to);
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

// Chunk c's slots to their places: thread (p, e) sums expert e's counts over
// the chunks c' = p mod parts, all of them and those before c.
__global__ __launch_bounds__(kRouteThreads) void k_route_place(const int *__restrict__ ids,
                                                              const int *__restrict__ counts,
                                                              int *__restrict__ offsets,
                                                              int *__restrict__ order, int T, int E,
                                                              int top_k, int chunk, int chunks,
                                                              int bits)
{
    __shared__ RouteLds l;
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

hipError_t launch_route(const float *logits, int *ids, float *weights, int *offsets, int *order,
                        void *workspace, int T, int E, int top_k, bool renorm, hipStream_t st)
{
    const int chunk = route_chunk(T), chunks = route_chunks(T);
    int *counts = chunks > 1 ? static_cast<int *>(workspace) : nullptr;
    int bits = 0;
    while ((1 << bits) < E)
        ++bits;
    auto kernel = E <= 64 ? k_route<1> : E <= 128 ? k_route<2> : E <= 256 ? k_route<4> : k_route<16>;
    hipError_t e = launch_kernel(kernel, dim3((unsigned)chunks), dim3(kRouteThreads), 0, st, logits,
                                 ids, weights, offsets, order, counts, T, E, top_k, renorm ? 1 : 0,
                                 chunk, bits);
    if (e != hipSuccess || !counts)
        return e;
    return launch_kernel(k_route_place, dim3((unsigned)chunks), dim3(kRouteThreads), 0, st,
                         (const int *)ids, (const int *)counts, offsets, order, T, E, top_k, chunk,
                         chunks, bits);
}

}  // namespace q4k
