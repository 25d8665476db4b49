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
//
// Bound by the logits' bytes: 509 x 163840 in fp32 without a list 60 us (5.6
// TB/s), with the 8 largest 63 to 67, the 20 largest 79: the list's steps, ballots and a barrier, stand
// between a block's loads and its end, and the join takes 5. A thread holds 16
// or 32 elements (64 were slower: fewer blocks on a CU, loads behind each other),
// read by loads of 16 bytes where a row allows it; each element costs a
// difference, a product, an exponential, a clamp, two sums and half an operation
// for the maximum, which half the bytes do not hide: 509 x 163840 in bf16 37 us
// without a list (4.5 TB/s; vector operations issue in every cycle), with the 8
// largest 59. Rows that are equal in most places, as a grammar's mask leaves them,
// reach the bound everywhere and are taken one by one: 173 us with 163000 of the
// 163840 banned.
// One row: 7.5 us and the join's 4.6, the latencies of two short kernels.
#include "k3moe_internal.h"
#include "k3moe_device.h"

namespace k3moe {
namespace {

constexpr int kLpThreads = 256, kLpWaves = kLpThreads / 64;
constexpr int kLpMaxTop = 64, kLpCand = 1024;
constexpr int kLpMaxVocab = 1 << 24, kLpMaxIds = 4096;
constexpr int kLpShort = 16, kLpLong = 32;   // elements per thread

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

// Wave reductions through DPP, the result in every lane (read back from lane 63).
template <class T, class F>
__device__ __forceinline__ T lp_wave(T v, T none, F f)
{
    auto step = [&](auto ctrl, auto rows) {
        constexpr int kCtrl = decltype(ctrl)::value, kRows = decltype(rows)::value;
        uint32_t w[sizeof(T) / 4], n[sizeof(T) / 4];
        __builtin_memcpy(w, &v, sizeof(T));
        __builtin_memcpy(n, &none, sizeof(T));
#pragma unroll
        for (unsigned i = 0; i < sizeof(T) / 4; ++i)
            w[i] = (uint32_t)__builtin_amdgcn_update_dpp((int)n[i], (int)w[i], kCtrl, kRows, 0xf, false);
        T x;
        __builtin_memcpy(&x, w, sizeof(T));
        v = f(v, x);
    };
    typedef std::integral_constant<int, 0xf> all;
    step(std::integral_constant<int, 0xb1>{}, all{});                                   // neighbours
    step(std::integral_constant<int, 0x4e>{}, all{});                                   // pairs
    step(std::integral_constant<int, 0x141>{}, all{});                                  // half rows
    step(std::integral_constant<int, 0x140>{}, all{});                                  // rows
    step(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xa>{});     // row 0 into 1, 2 into 3
    step(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xc>{});     // row 1 into 2 and 3
    uint32_t w[sizeof(T) / 4];
    __builtin_memcpy(w, &v, sizeof(T));
#pragma unroll
    for (unsigned i = 0; i < sizeof(T) / 4; ++i) w[i] = (uint32_t)__builtin_amdgcn_readlane((int)w[i], 63);
    T r;
    __builtin_memcpy(&r, w, sizeof(T));
    return r;
}

struct LpMax {
    template <class T>
    __device__ __forceinline__ T operator()(T a, T b) const { return a > b ? a : b; }
};
struct LpFmax {   // passes over NaN
    __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct LpAdd {
    template <class T>
    __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};

// Joins a block's waves; red: one place per wave. W waves.
template <int W, class T, class F>
__device__ __forceinline__ T lp_block(T v, T none, T *red, F f)
{
    v = lp_wave(v, none, f);
    if constexpr (W > 1) {
        __syncthreads();             // what was in red is read
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int w = 1; w < W; ++w) v = f(v, red[w]);
    }
    return v;
}

// A bound that at least k of the wave's elements reach, as the key of a logit: the k-th largest of the lanes' maxima,
// rounded down to its first 22 bits. 0 where fewer than k lanes hold any.
__device__ __forceinline__ uint32_t lp_bound(uint32_t best, int k)
{
    uint32_t tau = 0u;
#pragma unroll
    for (int b = 31; b >= 10; --b) {
        const uint32_t c = tau | (1u << b);
        if (__popcll(__ballot(best >= c)) >= k) tau = c;
    }
    return tau;
}

struct LpTop {
    uint64_t list[kLpCand], red[kLpWaves];
    int count;
};

// The k largest of the keys that a block's threads hold, all that reach a bound (which k of them do) being in L.list,
// L.count of them. each(f): calls f(key) for all of this thread's keys; put(rank, key), key 0: there is none. Every
// thread of the block calls it. W waves.
template <int W, class Each, class Put>
__device__ __forceinline__ void lp_rank(LpTop &L, int k, Each each, Put put)
{
    const int tid = threadIdx.x, n = L.count;
    if (n <= kLpCand) {
        for (int i = tid; i < n; i += 64 * W) {
            const uint64_t key = L.list[i];
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += L.list[j] > key ? 1 : 0;
            if (rank < k) put(rank, key);
        }
        for (int i = n + tid; i < k; i += 64 * W) put(i, 0ull);
    } else {
        uint64_t last = ~0ull;
        for (int r = 0; r < k; ++r) {
            uint64_t next = 0ull;
            each([&](uint64_t key) { next = key < last && key > next ? key : next; });
            next = lp_block<W, uint64_t>(next, 0ull, L.red, LpMax());
            if (tid == 0) put(r, next);
            last = next;
        }
    }
}

__device__ __forceinline__ void lp_collect(LpTop &L, uint64_t key)
{
    const int at = atomicAdd(&L.count, 1);   // the order of the list does not matter: every key has its own rank
    if (at < kLpCand) L.list[at] = key;
}

// One chunk of VPT * 256 logits of a row. W: neighbouring elements per load.
template <int VPT, bool F32, int W>
__global__ __launch_bounds__(kLpThreads, 6) void k_lp_chunk(LpParams p)
{
    __shared__ LpTop L;
    __shared__ float wmax[kLpWaves];
    __shared__ LpStats wsum[kLpWaves];
    __shared__ uint32_t wbound[kLpWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int t = blockIdx.x / p.chunks, c = blockIdx.x - t * p.chunks;
    const int base = c * VPT * kLpThreads;
    auto index = [&](int j) { return base + ((j / W) * kLpThreads + tid) * W + j % W; };

    float v[VPT];
    const int64_t row = (int64_t)t * p.stride;
    const bool whole = base + VPT * kLpThreads <= p.V;
    auto one = [&](int i) {
        return F32 ? static_cast<const float *>(p.x)[row + i] : bf16f(static_cast<const uint16_t *>(p.x)[row + i]);
    };
    if (whole) {
#pragma unroll
        for (int j = 0; j < VPT; j += W) {
            if constexpr (W == 1) {
                v[j] = one(index(j));
            } else if constexpr (F32) {
                const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.x) + row + index(j));
                v[j] = a.x, v[j + 1] = a.y, v[j + 2] = a.z, v[j + 3] = a.w;
            } else {
                const u4 a = *reinterpret_cast<const u4 *>(static_cast<const uint16_t *>(p.x) + row + index(j));
#pragma unroll
                for (int e = 0; e < 4; ++e) v[j + 2 * e] = bf16f(a[e] & 0xffffu), v[j + 2 * e + 1] = bf16f(a[e] >> 16);
            }
        }
    } else {   // a row's end, one by one
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const float x = one(min(index(j), p.V - 1));
            v[j] = index(j) < p.V ? x : -INFINITY;
        }
    }
    float group[VPT / 8], mine = -INFINITY;          // maxima of eight elements each; they pass over NaN
#pragma unroll
    for (int g = 0; g < VPT / 8; ++g) {
        group[g] = fmaxf(v[8 * g], v[8 * g + 1]);
#pragma unroll
        for (int j = 2; j < 8; j += 2) group[g] = fmaxf(fmaxf(group[g], v[8 * g + j]), v[8 * g + j + 1]);
        mine = fmaxf(mine, group[g]);
    }
    // lanes without an element hold none of the chunk's largest
    const float wm = lp_wave(mine, -INFINITY, LpFmax());
    const uint32_t key = index(0) < p.V ? order_key(mine + 0.0f) : 0u;
    if (lane == 0) wmax[wave] = wm;
    if (p.k > 0) {
        const uint32_t bound = lp_bound(key, p.k);
        if (lane == 0) wbound[wave] = bound;
    }
    if (tid == 0) L.count = 0;
    __syncthreads();
    float m = wmax[0];
#pragma unroll
    for (int w = 1; w < kLpWaves; ++w) m = fmaxf(m, wmax[w]);
    // e^(x - m) = 2^((x - m) L). The difference comes first: it is exact next to the maximum and keeps its digits at any
    // level, where x L - m L would lose |m| 2^-24 and overflow at masks of the type's lowest number.
    constexpr float L2E = 1.44269502f;
    const float use = m == -INFINITY ? 0.0f : m;
    float rest = 0.0f, dev = 0.0f;                   // sums of e and of (m - x) L e
    int top = 0;
    // -inf: e is 0, and so is its term of the deviation; +inf: x - m is NaN and stays
    if (wm == m && m < INFINITY) {         // the wave that holds the maximum counts it apart
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const float t = (v[j] - use) * L2E, e = __builtin_amdgcn_exp2f(t);
            const bool peak = v[j] == m;
            top += peak ? 1 : 0;
            rest += peak ? 0.0f : e;
            dev = fmaf(-fmaxf(t, -512.0f), e, dev);  // the maximum's own t is 0
        }
        if (m == -INFINITY) top = 0, rest = rest != rest ? rest : 0.0f;
    } else {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const float t = (v[j] - use) * L2E, e = __builtin_amdgcn_exp2f(t);
            rest += e;
            dev = fmaf(-fmaxf(t, -512.0f), e, dev);
        }
    }
    {
        const double R = lp_wave<double>(rest, 0.0, LpAdd()), D = lp_wave<double>(dev, 0.0, LpAdd());
        const int N = lp_wave<int>(top, 0, LpAdd());
        if (lane == 0) wsum[wave] = LpStats{R, D * (1.0 / (double)L2E), m, N};
    }
    if (p.k > 0) {
        uint32_t bound = wbound[0];
#pragma unroll
        for (int w = 1; w < kLpWaves; ++w) bound = max(bound, wbound[w]);
        if (__ballot(key >= bound && key)) {
            // -inf and NaN, which rank alike, are among the largest only of a chunk with few others
            const bool low = bound <= order_key(-INFINITY);
            const float least = low ? -INFINITY : __uint_as_float(bound & 0x80000000u ? bound ^ 0x80000000u : ~bound);
#pragma unroll
            for (int g = 0; g < VPT / 8; ++g) {
                if (__ballot(low || group[g] >= least)) {
#pragma unroll
                    for (int j = 8 * g; j < 8 * g + 8; ++j) {
                        const int i = index(j);
                        if ((low || v[j] >= least) && i < p.V) lp_collect(L, lp_key(v[j], i));
                    }
                }
            }
        }
    }
    __syncthreads();
    if (tid == 0) {
        LpStats s = wsum[0];
#pragma unroll
        for (int w = 1; w < kLpWaves; ++w) s.rest += wsum[w].rest, s.dev += wsum[w].dev, s.top += wsum[w].top;
        p.stats[(int64_t)t * p.chunks + c] = s;
    }
    if (p.k == 0) return;
    uint64_t *out = p.cand + ((int64_t)t * p.chunks + c) * p.k;
    lp_rank<kLpWaves>(L, p.k,
                      [&](auto f) {
#pragma unroll
                          for (int j = 0; j < VPT; ++j) {
                              const int i = index(j);
                              if (i < p.V) f(lp_key(v[j], i));
                          }
                      },
                      [&](int rank, uint64_t key) { out[rank] = key; });
}

// Joins a row's chunks: one block of W waves per row, whose threads hold the chunks' candidates, up to 64 W CPT of them
// (CPT 0: any number, read again where they are needed). Everything that does not wait for the sums is loaded first.
template <bool F32, int W, int CPT>
__global__ __launch_bounds__(64 * W) void k_lp_join(LpParams p)
{
    __shared__ LpTop L;
    const int tid = threadIdx.x, t = blockIdx.x;
    const LpStats *st = p.stats + (int64_t)t * p.chunks;
    const uint64_t *cand = p.cand + (int64_t)t * p.chunks * p.k;
    const int n = p.chunks * p.k;
    const LpStats mine = tid < p.chunks ? st[tid] : LpStats{0.0, 0.0, -INFINITY, 0};
    const int64_t ids0 = (int64_t)t * p.n_ids;
    const int id0 = tid < p.n_ids ? p.ids[ids0 + tid] : -1;
    uint64_t held[CPT > 0 ? CPT : 1];
    uint64_t best = 0ull;
    if constexpr (CPT > 0) {
#pragma unroll
        for (int i = 0; i < CPT; ++i) held[i] = tid + 64 * W * i < n ? cand[tid + 64 * W * i] : 0ull;
    }
    const float x0 = id0 >= 0 && id0 < p.V ? lp_logit(p, F32, t, id0) : NAN;
    auto each = [&](auto f) {
        if constexpr (CPT > 0) {
#pragma unroll
            for (int i = 0; i < CPT; ++i) f(held[i]);
        } else {
            for (int i = tid; i < n; i += 64 * W) f(cand[i]);
        }
    };
    each([&](uint64_t key) { best = key > best ? key : best; });
    float m = mine.m;
    for (int c = tid + 64 * W; c < p.chunks; c += 64 * W) m = fmaxf(m, st[c].m);
    m = lp_block<W, float>(m, -INFINITY, reinterpret_cast<float *>(L.red), LpFmax());
    double s = 0.0, dev = 0.0;
    int top = 0;
    auto add = [&](const LpStats &x) {
        const double part = x.rest + x.top;
        if (x.m == m) {
            s += x.rest, dev += x.dev, top += x.top;
        } else if (part != 0.0) {          // else nothing but -inf
            const double f = exp((double)x.m - (double)m);
            s += part * f, dev += f * (x.dev + ((double)m - (double)x.m) * part);
        }
    };
    add(mine);
    for (int c = tid + 64 * W; c < p.chunks; c += 64 * W) add(st[c]);
    s = lp_block<W, double>(s, 0.0, reinterpret_cast<double *>(L.red), LpAdd());
    dev = lp_block<W, double>(dev, 0.0, reinterpret_cast<double *>(L.red), LpAdd());
    top = lp_block<W, int>(top, 0, reinterpret_cast<int *>(L.red), LpAdd());
    // no maximum that counts: a row of -inf, of NaN, or with +inf
    const double log_s = top > 0 ? log1p(s + (top - 1)) : (double)NAN;
    const double peak = (double)m;
    if (p.ent && tid == 0) p.ent[t] = (float)(log_s + dev / (s + top));
    if (tid < p.n_ids) p.lp[ids0 + tid] = (float)((double)x0 - peak - log_s);
    for (int j = tid + 64 * W; j < p.n_ids; j += 64 * W) {
        const int i = p.ids[ids0 + j];
        p.lp[ids0 + j] = i >= 0 && i < p.V ? (float)((double)lp_logit(p, F32, t, i) - peak - log_s) : NAN;
    }
    if (p.k == 0) return;
    if (tid == 0) L.count = 0;
    const uint32_t bound = lp_block<W, uint32_t>(lp_bound((uint32_t)(best >> 32), p.k), 0u, reinterpret_cast<uint32_t *>(L.red), LpMax());
    __syncthreads();
    if ((uint32_t)(best >> 32) >= bound)
        each([&](uint64_t key) {
            if (key && (uint32_t)(key >> 32) >= bound) lp_collect(L, key);
        });
    __syncthreads();
    lp_rank<W>(L, p.k, each, [&](int rank, uint64_t key) {
        const int64_t o = (int64_t)t * p.k + rank;
        const uint32_t b = (uint32_t)(key >> 32), v = b & 0x80000000u ? b ^ 0x80000000u : ~b;   // the logit of the key
        p.top_ids[o] = (int)~(uint32_t)key;
        p.top_lp[o] = (float)((double)__uint_as_float(v) - peak - log_s);
    });
}

// Chunks of a row: long ones where they still give every CU some blocks (a chunk's ends, the top list first of all,
// cost the same for both). Short and long, rows x 163840, k = 20: 1: 11.9 and 13.5 us, 16: 13.7 and 14.7, 32 (640 long
// chunks): 15.8 and 15.6, 64: 23.2 and 21.8, 509: 96 and 80; 128 x 32000 (512): 12.4 and 13.4.
constexpr int64_t kLpLongFrom = 640;
int64_t lp_long_chunks(int64_t V) { return (V + kLpLong * kLpThreads - 1) / (kLpLong * kLpThreads); }
int lp_per_thread(int64_t T, int64_t V) { return T * lp_long_chunks(V) >= kLpLongFrom ? kLpLong : kLpShort; }
int lp_chunks(int64_t T, int64_t V)
{
    const int64_t per = (int64_t)lp_per_thread(T, V) * kLpThreads;
    return (int)((V + per - 1) / per);
}
size_t lp_stat_bytes(int64_t T, int64_t V) { return ((size_t)(T * lp_chunks(T, V)) * sizeof(LpStats) + 255) / 256 * 256; }
size_t lp_bytes(int64_t T, int64_t V, int k) { return lp_stat_bytes(T, V) + (size_t)(T * lp_chunks(T, V)) * (size_t)k * 8; }
// The most that T rows or fewer take: the largest number of rows in short chunks may take more than T in long ones.
size_t lp_most_bytes(int64_t T, int64_t V, int k)
{
    const int64_t shorts = min(T, (kLpLongFrom - 1) / lp_long_chunks(V));
    return max(lp_bytes(T, V, k), lp_bytes(shorts, V, k));
}

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
    const int64_t cand = p.chunks * (int64_t)p.k;
    if (cand <= 256) k_lp_join<F32, 1, 4><<<(unsigned)p.T, 64, 0, s>>>(p);
    else if (cand <= 1024) k_lp_join<F32, kLpWaves, 4><<<(unsigned)p.T, kLpThreads, 0, s>>>(p);
    else k_lp_join<F32, kLpWaves, 0><<<(unsigned)p.T, kLpThreads, 0, s>>>(p);
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
    if (st == K3MOE_OK) *bytes = lp_most_bytes(T, V, k);
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
