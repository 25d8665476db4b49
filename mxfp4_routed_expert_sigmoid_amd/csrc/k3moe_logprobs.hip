// Log probabilities (k3moe_logprobs). Per row x of V logits, with m = max x:
//   s = sum e^(x - m),  lp(i) = x_i - m - log s,
//   entropy = log s + sum (m - x) e^(x - m) / s
// (both terms of the entropy are >= 0: nothing cancels), and the k largest.
//
// One pass over the logits: a block takes a chunk of a row into registers and
// leaves its maximum, its two sums and its k largest; a second kernel joins a
// row's chunks, in their order, in 64 bits. The maximum's own e^0 is counted
// apart from the sum of the others: a row that is nearly sure of one token keeps
// the digits of what is left.
//
// The k largest of a chunk: every wave finds the k-th largest of its 64 lanes'
// maxima by ballots, the block takes the largest of these as a bound that k of
// its elements reach, and ranks what reaches it. Where too much does (many equal
// logits) it takes the elements one by one instead.
#include "k3moe_internal.h"
#include "k3moe_device.h"

namespace k3moe {
namespace {

constexpr int kLpThreads = 256, kLpWaves = kLpThreads / 64;
constexpr int kLpMaxTop = 64, kLpCand = 1024;
constexpr int kLpMaxVocab = 1 << 24, kLpMaxIds = 4096;
constexpr int kLpShort = 16, kLpLong = 64;   // elements per thread

struct LpStats {
    double rest, dev;   // sum of e^(x - m) but for the maxima, sum of (m - x) e^(x - m)
    float m;
    int top;            // elements equal to m
};

struct LpParams {
    const void *x;
    int64_t stride;
    int T, V, chunks, k, n_ids;
    const int32_t *ids;
    float *lp, *ent, *top_lp;
    int32_t *top_ids;
    LpStats *stats;      // [T][chunks]
    uint64_t *cand;      // [T][chunks][k], a chunk's largest first, 0: none
};

// The order of the top list in one word: larger logits first, equal ones (the two zeros too) by their number. 0 is no
// element.
__device__ __forceinline__ uint64_t lp_key(float v, int i) { return ((uint64_t)order_key(v + 0.0f) << 32) | (uint32_t)~(uint32_t)i; }

__device__ __forceinline__ float lp_logit(const LpParams &p, bool f32, int t, int i)
{
    const int64_t o = (int64_t)t * p.stride + i;
    return f32 ? static_cast<const float *>(p.x)[o] : bf16f(static_cast<const uint16_t *>(p.x)[o]);
}

// e^d for d <= 0, to about an ulp: the product with log2(e) is held in two parts.
__device__ __forceinline__ float lp_exp(float d)
{
    const float t = d * 1.44269502f, e = fmaf(d, 1.44269502f, -t) + d * 1.92596299e-8f;
    const float x = __builtin_amdgcn_exp2f(t);
    return d < -126.0f * 0.69314718f ? x : fmaf(x, e * 0.69314718f, x);
}

template <class T, class F>
__device__ __forceinline__ T block_reduce(T v, T *red, F f)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = f(v, __shfl_xor(v, o));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < kLpWaves; ++w) v = f(v, red[w]);
    return v;
}

// The k largest of the keys that the block's threads hold. best: this thread's largest (0: none); each(f): calls
// f(key) for all of its keys; put(rank, key). Every thread of the block calls it.
template <class Each, class Put>
__device__ __forceinline__ void block_top(uint64_t best, int k, uint64_t *list, int *count, uint64_t *red, Each each, Put put)
{
    const int tid = threadIdx.x;
    // the k-th largest of the wave's 64 maxima (0 where fewer lanes hold any)
    const uint32_t mine = (uint32_t)(best >> 32);
    uint32_t tau = 0u;
#pragma unroll
    for (int b = 31; b >= 0; --b) {
        const uint32_t c = tau | (1u << b);
        if (__popcll(__ballot(mine >= c)) >= k) tau = c;
    }
    if (tid == 0) *count = 0;
    const uint64_t bound = block_reduce<uint64_t>((uint64_t)tau << 32, red, [](uint64_t a, uint64_t b) { return a > b ? a : b; });
    each([&](uint64_t key) {
        if (key >= bound && key) {
            const int at = atomicAdd(count, 1);   // the order of the list does not matter: every key has its own rank
            if (at < kLpCand) list[at] = key;
        }
    });
    __syncthreads();
    const int n = *count;
    if (n <= kLpCand) {
        for (int i = tid; i < n; i += kLpThreads) {
            const uint64_t key = list[i];
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += list[j] > key ? 1 : 0;
            if (rank < k) put(rank, key);
        }
        for (int i = n + tid; i < k; i += kLpThreads) put(i, 0ull);
    } else {
        uint64_t last = ~0ull;
        for (int r = 0; r < k; ++r) {
            uint64_t next = 0ull;
            each([&](uint64_t key) { next = key < last && key > next ? key : next; });
            next = block_reduce<uint64_t>(next, red, [](uint64_t a, uint64_t b) { return a > b ? a : b; });
            if (tid == 0) put(r, next);
            last = next;
        }
    }
}

// One chunk of VPT * 256 logits of a row. W: neighbouring elements per load.
template <int VPT, bool F32, int W>
__global__ __launch_bounds__(kLpThreads) void k_lp_chunk(LpParams p)
{
    __shared__ uint64_t list[kLpCand], red[kLpWaves];
    __shared__ int count;
    const int tid = threadIdx.x;
    const int t = blockIdx.x / p.chunks, c = blockIdx.x - t * p.chunks;
    const int base = c * VPT * kLpThreads;
    auto index = [&](int j) { return base + ((j / W) * kLpThreads + tid) * W + j % W; };

    float v[VPT];
    const int64_t row = (int64_t)t * p.stride;
#pragma unroll
    for (int j = 0; j < VPT; j += W) {
        const int i = min(index(j), p.V - 1) / W * W;   // a last load that ends behind the row is shortened below
        if constexpr (W == 1) {
            v[j] = F32 ? static_cast<const float *>(p.x)[row + i] : bf16f(static_cast<const uint16_t *>(p.x)[row + i]);
        } else if constexpr (F32) {
            if (i + W <= p.V) {
                const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.x) + row + i);
                v[j] = a.x, v[j + 1] = a.y, v[j + 2] = a.z, v[j + 3] = a.w;
            } else {
#pragma unroll
                for (int e = 0; e < W; ++e) v[j + e] = static_cast<const float *>(p.x)[row + min(i + e, p.V - 1)];
            }
        } else {
            if (i + W <= p.V) {
                const u4 a = *reinterpret_cast<const u4 *>(static_cast<const uint16_t *>(p.x) + row + i);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[j + 2 * e] = bf16f(a[e] & 0xffffu), v[j + 2 * e + 1] = bf16f(a[e] >> 16);
            } else {
#pragma unroll
                for (int e = 0; e < W; ++e) v[j + e] = bf16f(static_cast<const uint16_t *>(p.x)[row + min(i + e, p.V - 1)]);
            }
        }
    }
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        if (index(j) >= p.V) v[j] = -INFINITY;
        m = fmaxf(m, v[j]);          // passes over NaN
    }
    m = block_reduce<float>(m, reinterpret_cast<float *>(red), [](float a, float b) { return fmaxf(a, b); });
    const float use = m == -INFINITY ? 0.0f : m;
    float rest = 0.0f, dev = 0.0f;
    int top = 0;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const float d = v[j] - use, e = lp_exp(d);
        const bool peak = v[j] == m && m != -INFINITY;
        top += peak && m < INFINITY ? 1 : 0;
        rest += peak && m < INFINITY ? 0.0f : e;       // +inf: d is NaN and stays
        dev -= e == 0.0f ? 0.0f : d * e;
    }
    const double R = block_reduce<double>(rest, reinterpret_cast<double *>(red), [](double a, double b) { return a + b; });
    const double Dv = block_reduce<double>(dev, reinterpret_cast<double *>(red), [](double a, double b) { return a + b; });
    const int N = block_reduce<int>(top, reinterpret_cast<int *>(red), [](int a, int b) { return a + b; });
    if (tid == 0) p.stats[(int64_t)t * p.chunks + c] = LpStats{R, Dv, m, N};
    if (p.k == 0) return;

    uint64_t best = 0ull;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = index(j);
        const uint64_t key = i < p.V ? lp_key(v[j], i) : 0ull;
        best = key > best ? key : best;
    }
    uint64_t *out = p.cand + ((int64_t)t * p.chunks + c) * p.k;
    block_top(best, p.k, list, &count, red,
              [&](auto f) {
#pragma unroll
                  for (int j = 0; j < VPT; ++j) {
                      const int i = index(j);
                      if (i < p.V) f(lp_key(v[j], i));
                  }
              },
              [&](int rank, uint64_t key) { out[rank] = key; });
}

// Joins a row's chunks: one block per row.
template <bool F32>
__global__ __launch_bounds__(kLpThreads) void k_lp_join(LpParams p)
{
    __shared__ uint64_t list[kLpCand], red[kLpWaves];
    __shared__ int count;
    const int tid = threadIdx.x, t = blockIdx.x;
    const LpStats *st = p.stats + (int64_t)t * p.chunks;
    float m = -INFINITY;
    for (int c = tid; c < p.chunks; c += kLpThreads) m = fmaxf(m, st[c].m);
    m = block_reduce<float>(m, reinterpret_cast<float *>(red), [](float a, float b) { return fmaxf(a, b); });
    double s = 0.0, dev = 0.0;
    for (int c = tid; c < p.chunks; c += kLpThreads) {
        const LpStats x = st[c];
        const double part = x.rest + x.top;
        if (part == 0.0) continue;       // nothing but -inf
        const double f = x.m == m ? 1.0 : exp((double)x.m - (double)m);
        s += x.m == m ? x.rest : part * f;
        dev += f * (x.dev + (x.m == m ? 0.0 : ((double)m - (double)x.m) * part));
    }
    int top = 0;
    for (int c = tid; c < p.chunks; c += kLpThreads) top += st[c].m == m ? st[c].top : 0;
    s = block_reduce<double>(s, reinterpret_cast<double *>(red), [](double a, double b) { return a + b; });
    dev = block_reduce<double>(dev, reinterpret_cast<double *>(red), [](double a, double b) { return a + b; });
    top = block_reduce<int>(top, reinterpret_cast<int *>(red), [](int a, int b) { return a + b; });
    // no maximum that counts: a row of -inf, of NaN, or with +inf
    const double log_s = top > 0 ? log1p(s + (top - 1)) : (double)NAN;
    const double peak = (double)m;
    if (p.ent && tid == 0) p.ent[t] = (float)(log_s + dev / (s + top));
    for (int j = tid; j < p.n_ids; j += kLpThreads) {
        const int64_t o = (int64_t)t * p.n_ids + j;
        const int i = p.ids[o];
        p.lp[o] = i >= 0 && i < p.V ? (float)((double)lp_logit(p, F32, t, i) - peak - log_s) : NAN;
    }
    if (p.k == 0) return;
    const uint64_t *cand = p.cand + (int64_t)t * p.chunks * p.k;
    const int n = p.chunks * p.k;
    uint64_t best = 0ull;
    for (int i = tid; i < n; i += kLpThreads) best = cand[i] > best ? cand[i] : best;
    block_top(best, p.k, list, &count, red,
              [&](auto f) {
                  for (int i = tid; i < n; i += kLpThreads) f(cand[i]);
              },
              [&](int rank, uint64_t key) {
                  const int i = (int)~(uint32_t)key;
                  const int64_t o = (int64_t)t * p.k + rank;
                  p.top_ids[o] = i;
                  p.top_lp[o] = (float)((double)lp_logit(p, F32, t, i) - peak - log_s);
              });
}

// Chunks of a row: long ones where they still give every CU some blocks (a chunk's ends, the top list first of all,
// cost the same for both).
int lp_per_thread(int64_t T, int64_t V)
{
    return T * ((V + kLpLong * kLpThreads - 1) / (kLpLong * kLpThreads)) >= 512 ? kLpLong : kLpShort;
}
int lp_chunks(int64_t T, int64_t V)
{
    const int64_t per = (int64_t)lp_per_thread(T, V) * kLpThreads;
    return (int)((V + per - 1) / per);
}
size_t lp_stat_bytes(int64_t T, int64_t V) { return ((size_t)(T * lp_chunks(T, V)) * sizeof(LpStats) + 255) / 256 * 256; }
size_t lp_bytes(int64_t T, int64_t V, int k) { return lp_stat_bytes(T, V) + (size_t)(T * lp_chunks(T, V)) * (size_t)k * 8; }

template <bool F32>
void launch_lp(const LpParams &p, bool vec, hipStream_t s)
{
    constexpr int W = F32 ? 4 : 8;
    const unsigned grid = (unsigned)((int64_t)p.T * p.chunks);
    if (lp_per_thread(p.T, p.V) == kLpLong) {
        if (vec) k_lp_chunk<kLpLong, F32, W><<<grid, kLpThreads, 0, s>>>(p);
        else k_lp_chunk<kLpLong, F32, 1><<<grid, kLpThreads, 0, s>>>(p);
    } else {
        if (vec) k_lp_chunk<kLpShort, F32, W><<<grid, kLpThreads, 0, s>>>(p);
        else k_lp_chunk<kLpShort, F32, 1><<<grid, kLpThreads, 0, s>>>(p);
    }
    k_lp_join<F32><<<(unsigned)p.T, kLpThreads, 0, s>>>(p);
}

bool at(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

k3moe_status lp_sizes(int32_t T, int32_t V, int32_t k)
{
    if (T < 0 || V <= 0 || k < 0 || k > V) return K3MOE_E_INVALID_ARG;
    // blocks, and a row's work-items, are counted in 32 bits
    if (V > kLpMaxVocab || k > kLpMaxTop || (int64_t)T * lp_chunks(T, V) >= (int64_t)1 << 24) return K3MOE_E_UNSUPPORTED_SHAPE;
    return K3MOE_OK;
}

}  // namespace
}  // namespace k3moe

using namespace k3moe;

extern "C" k3moe_status k3moe_logprobs_workspace_size(int32_t T, int32_t V, int32_t k, size_t *bytes)
{
    if (!bytes) return K3MOE_E_INVALID_ARG;
    const k3moe_status st = lp_sizes(T, V, k);
    if (st == K3MOE_OK) *bytes = lp_bytes(T, V, k);
    return st;
}

extern "C" k3moe_status k3moe_logprobs(const void *logits, int32_t logits_f32, int64_t stride, int32_t T, int32_t V,
                                       const int32_t *ids, int32_t n_ids, float *lp, float *entropy, int32_t *top_ids,
                                       float *top_lp, int32_t k, void *workspace, size_t workspace_bytes, void *stream)
{
    if (logits_f32 < 0 || logits_f32 > 1 || n_ids < 0) return K3MOE_E_INVALID_ARG;
    if (const k3moe_status st = lp_sizes(T, V, k); st != K3MOE_OK) return st;
    if (n_ids > kLpMaxIds) return K3MOE_E_UNSUPPORTED_SHAPE;
    if (T == 0) return K3MOE_OK;
    if (!logits || (ids != nullptr) != (n_ids > 0) || (lp != nullptr) != (n_ids > 0) || (top_ids != nullptr) != (k > 0) ||
        (top_lp != nullptr) != (k > 0) || (!lp && !entropy && !top_ids))
        return K3MOE_E_INVALID_ARG;
    if (T == 1) stride = V;
    if (stride < V) return K3MOE_E_INVALID_ARG;
    if (!at(logits, logits_f32 ? 4 : 2) || !at(ids, 4) || !at(lp, 4) || !at(entropy, 4) || !at(top_ids, 4) || !at(top_lp, 4))
        return K3MOE_E_ALIGNMENT;
    if (!workspace || !at(workspace, 256) || workspace_bytes < lp_bytes(T, V, k)) return K3MOE_E_WORKSPACE;
    LpParams p{};
    p.x = logits, p.stride = stride, p.T = T, p.V = V, p.chunks = lp_chunks(T, V), p.k = k, p.n_ids = n_ids;
    p.ids = ids, p.lp = lp, p.ent = entropy, p.top_ids = top_ids, p.top_lp = top_lp;
    p.stats = static_cast<LpStats *>(workspace);
    p.cand = reinterpret_cast<uint64_t *>(static_cast<uint8_t *>(workspace) + lp_stat_bytes(T, V));
    const bool vec = at(logits, 16) && (T == 1 || stride % (logits_f32 ? 4 : 8) == 0);
    hipStream_t s = static_cast<hipStream_t>(stream);
    logits_f32 ? launch_lp<true>(p, vec, s) : launch_lp<false>(p, vec, s);
    return hipGetLastError() == hipSuccess ? K3MOE_OK : K3MOE_E_HIP;
}
