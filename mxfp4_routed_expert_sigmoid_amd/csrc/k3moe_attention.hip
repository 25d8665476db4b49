// Attention of packed sequences (k3moe_attention): per sequence, query head and
// query i of n over keys j of N
//   s_j = scale q_i . k_j,  out = sum_j e^(s_j) v_j / sum_j e^(s_j),
//   lse = log sum_j e^(s_j),  causal: j <= i + N - n
// in one pass over the keys with the running maximum and sum.
//
// A block of four waves owns 128 queries of one head, a wave 32 of them
// (k3moe_attn.h). Tiles of 64 keys and values go through LDS by direct loads
// into two buffers, one barrier per tile. Where the tiles of queries are too few
// for the card their keys are split over blocks, whose unnormalised sums a second
// kernel joins in their order.
//
// Two blocks fit a CU (64 KB of LDS and 256 registers a lane at heads of 128), so
// one's barrier and masked tiles stand in the other's products. Whole tiles and
// those on the diagonal or at the end take loops of their own: the accumulators
// then stay where they are. Bound by the matrix unit and the exponentials beside
// it (k3moe_attn.h): 8192 causal tokens of 32 heads of 128 550 to 580 us (0.95 to
// 1.0 PFLOP/s), heads of 64, 4096 tokens, 93 (0.74: the same exponentials for half
// the products), of 192 / 128, 16 heads, 115 (0.75: its registers spill a little
// outside the loop of whole tiles). Short prompts packed together (7 of 1 to 2047
// tokens, 32 heads) 76 to 88 us, 0.65 PFLOP/s: 1184 blocks of 1 to 32 tiles, of
// whose time first loads, masked tiles and last stores take a larger part.
#include "k3moe_attn.h"

namespace k3moe {
namespace {

constexpr int kPrWaves = 4, kPrRows = kPrWaves * kAtRows;
constexpr int kPrBlocks = 512;        // blocks that a split makes at most: two per CU
constexpr int kPrMaxSplit = 16, kPrLeast = 2;  // parts of a tile's keys, tiles of keys of a part at least
constexpr int kPrFrom = 6;            // tiles of keys that are split at least
constexpr int kPrGain = 28;           // what a tile of keys costs a block over what a part costs the launch, two per CU

struct PromptParams {
    const uint16_t *q, *k, *v;
    const int32_t *cu_q, *cu_k;
    uint16_t *out;
    float *lse, *part, *ml;   // part [tiles][heads][split][128][DV], ml the same of pairs
    int4 *joins;              // [tiles]: first query, queries, tile, tiles of keys, for the join
    int64_t qs, ks, vs, os;   // row strides, elements
    int seqs, Tq, Tk, Hq, group, causal, split;
    float scale;
};

// A tile of queries: its sequence's rows, its number there, and the tiles of keys that its last row sees.
struct PromptTile {
    int q0, n, k0, N, tile, keys;     // n: 0: there is no such tile
};

// Tiles in the order of the most keys first (in the sequences' order the last ones began late: 2 x 2048 tokens x 16
// heads 66 us, so 54). The tile's place in it, among 64 sequences at a time: the level, a number of tiles of
// keys, that the place falls in is found by halving, a lane counting the tiles of its sequence that reach it.
__device__ __forceinline__ PromptTile prompt_tile(const PromptParams &p, int place)
{
    const int lane = threadIdx.x & 63;
    const int32_t *cu_k = p.cu_k ? p.cu_k : p.cu_q;
    PromptTile r{};
    for (int b0 = 0; b0 < p.seqs; b0 += 64) {
        int lo = 0, hi = 0, klo = 0, khi = 0;
        if (b0 + lane < p.seqs) {
            lo = min(max(p.cu_q[b0 + lane], 0), p.Tq), klo = min(max(cu_k[b0 + lane], 0), p.Tk);
            hi = min(max(p.cu_q[b0 + lane + 1], lo), p.Tq), khi = min(max(cu_k[b0 + lane + 1], klo), p.Tk);
        }
        const int n = hi - lo, N = khi - klo, mine = (n + kPrRows - 1) / kPrRows;
        const int all = __builtin_amdgcn_readlane(wave_scan(mine), 63);
        if (place >= all) {
            place -= all;
            continue;
        }
        // this sequence's tiles with `level` tiles of keys or more: its last ones
        auto reach = [&](int level) {
            const int x = kAtKeys * (level - 1) - (p.causal ? N - n : 0);   // a tile's last row has to see more
            return level <= 0 ? mine : p.causal ? n <= x ? 0 : mine - max(x, 0) / kPrRows : N > x ? mine : 0;
        };
        int level = 0, above = p.Tk / kAtKeys + 2;   // reached by more tiles than `place`; not so
        int c = mine, next = 0;                                      // this sequence's tiles that reach either
        while (p.seqs > 1 && above - level > 1) {
            const int half = (level + above) >> 1, some = reach(half);
            if (__builtin_amdgcn_readlane(wave_scan(some), 63) > place) level = half, c = some;
            else above = half, next = some;
        }
        const int before = __builtin_amdgcn_readlane(wave_scan(next), 63), upto = wave_scan(c - next);
        const int at = __builtin_ctzll(__ballot(upto > place - before));
        r.q0 = __builtin_amdgcn_readlane(lo, at), r.n = __builtin_amdgcn_readlane(n, at);
        r.k0 = __builtin_amdgcn_readlane(klo, at), r.N = __builtin_amdgcn_readlane(N, at);
        r.tile = __builtin_amdgcn_readlane(mine - next - 1 - (place - before - (upto - (c - next))), at);
        const int see = p.causal ? min(kPrRows * (r.tile + 1), r.n) + r.N - r.n : r.N;
        r.keys = (max(see, 0) + kAtKeys - 1) / kAtKeys;
        return r;
    }
    return r;
}

// Tiles of keys of a part.
__device__ __forceinline__ int prompt_part(const PromptParams &p, int keys)
{
    return max((keys + p.split - 1) / p.split, kPrLeast);
}

template <int DK, int DV>
__global__ __launch_bounds__(64 * kPrWaves, 2) void k_attention(PromptParams p)
{
#ifdef __HIP_DEVICE_COMPILE__
    constexpr int KB = kAtKeys * DK * 2, VB = kAtKeys * DV * 2;
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5, l32 = lane & 31;
    const int head = blockIdx.x % p.Hq, unit = blockIdx.x / p.Hq, split = unit % p.split;
    const PromptTile x = prompt_tile(p, unit / p.split);
    const int n = x.n, N = x.N, per = prompt_part(p, x.keys);
    const int t0 = split * per, t1 = min(t0 + per, x.keys), tiles = t1 - t0;   // this part's tiles
    if (p.split > 1 && head == 0 && split == 0 && threadIdx.x == 0) p.joins[unit / p.split] = int4{x.q0, n, x.tile, x.keys};
    if (n == 0 || (split > 0 && tiles <= 0)) return;

    const int row = kPrRows * x.tile + kAtRows * wave + l32;   // this lane's query of the sequence
    AttRows<DK, DV> r;
    {
        const uint16_t *qp = p.q + (int64_t)(x.q0 + min(row, n - 1)) * p.qs + (int64_t)head * DK + 8 * h;
#pragma unroll
        for (int k = 0; k < DK / 16; ++k) r.q[k] = as_bf8(*reinterpret_cast<const u4 *>(qp + 16 * k));
    }
    r.clear();
    // keys that this lane's row and this wave's last row see, and that every row of the wave sees: the first ones
    const int see = p.causal ? min(row + 1 + N - n, N) : N;
    const int wfirst = kPrRows * x.tile + kAtRows * wave, wlast = min(wfirst + kAtRows, n) - 1;
    const int wsee = wfirst >= n ? 0 : p.causal ? wlast + 1 + N - n : N;
    const int wall = wfirst >= n ? 0 : p.causal ? wfirst + 1 + N - n : N;

    const int kvh = head / p.group;
    const uint16_t *kp = p.k + (int64_t)x.k0 * p.ks + (int64_t)kvh * DK, *vp = p.v + (int64_t)x.k0 * p.vs + (int64_t)kvh * DV;
    // Keys run a tile ahead of the values: tile t's scores are computed beside the weights of tile t - 1. i counts this
    // part's tiles.
    RowStage<DK, true> sk;
    RowStage<DV, false> sv;
    sk.init(p.ks), sv.init(p.vs);
    auto ktile = [&](int i) { return lds + (i & 1) * KB; };
    auto vtile = [&](int i) { return lds + 2 * KB + (i & 1) * VB; };
    // a wave loads 16 of a tile's rows; those behind the last key read as zeros
    auto load_k = [&](int i) {
        const int at = (t0 + i) * kAtKeys + 16 * wave;
        if (i < tiles) sk.load(kp + (int64_t)at * p.ks, p.ks, N - at, ktile(i) + 16 * wave * DK * 2);
    };
    auto load_v = [&](int i) {
        const int at = (t0 + i) * kAtKeys + 16 * wave;
        if (i < tiles) sv.load(vp + (int64_t)at * p.vs, p.vs, N - at, vtile(i) + 16 * wave * DV * 2);
    };
    const float c = p.scale * kLog2e;
    if (tiles > 0) {
        load_k(0), load_v(0), load_k(1);
        at_barrier();
        v16f s[2];
        att_scores(s, r, ktile(0));
        // every wave passes the same number of barriers, in whichever of the two loops
        const int pairs = max(min(wall / kAtKeys, t1) - t0, 0) / 2;
        int i = 0;
        float mx = pairs > 0 ? att_max(s) : 0.0f;
        for (; i < 2 * pairs; i += 2) {
            v16f o[2];
            at_barrier();
            load_k(i + 2), load_v(i + 1);
            att_tile(r, s, mx, o, lds + KB, vtile(0), c);
            at_barrier();
            load_k(i + 3), load_v(i + 2);
            att_tile(r, o, mx, s, lds, vtile(1), c);
        }
        for (; i < tiles; ++i) {
            at_barrier();
            load_k(i + 2), load_v(i + 1);
            const int first = (t0 + i) * kAtKeys;
            if (first < wsee) att_tile_masked(r, s, ktile(i + 1), vtile(i), c, low_bits(see - first), i + 1 < tiles);
        }
    }

    const float l = r.l + __shfl_xor(r.l, 32);
    if (row >= n) return;
    if (per >= x.keys) {          // one part
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        if (p.lse && h == 0)
            p.lse[(int64_t)(x.q0 + row) * p.Hq + head] = l == 0.0f ? -INFINITY : (r.m + __log2f(l)) * kLn2;
        uint16_t *op = p.out + (int64_t)(x.q0 + row) * p.os + (int64_t)head * DV + 4 * h;
#pragma unroll
        for (int d = 0; d < DV / 32; ++d)
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<uint2 *>(op + 32 * d + 2 * i) = uint2{at_pack(r.o[d][i] * inv, r.o[d][i + 1] * inv),
                                                                        at_pack(r.o[d][i + 2] * inv, r.o[d][i + 3] * inv)};
    } else {
        const int64_t at = (((int64_t)(unit / p.split) * p.Hq + head) * p.split + split) * kPrRows + kAtRows * wave + l32;
        float *op = p.part + at * DV + 4 * h;
#pragma unroll
        for (int d = 0; d < DV / 32; ++d)
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<float4 *>(op + 32 * d + 2 * i) = float4{r.o[d][i], r.o[d][i + 1], r.o[d][i + 2], r.o[d][i + 3]};
        if (h == 0) *reinterpret_cast<float2 *>(p.ml + 2 * at) = float2{r.m, l};
    }
#endif
}

// Joins the parts of a tile's keys: DV / 4 threads for a row.
template <int DV>
__global__ __launch_bounds__(256) void k_attention_join(PromptParams p)
{
    constexpr int TR = DV / 4, RB = 256 / TR;
    const int head = blockIdx.x % p.Hq, tile = blockIdx.x / p.Hq;
    const int4 d = p.joins[tile];
    const struct { int q0, n, tile, keys; } x = {d.x, d.y, d.z, d.w};
    const int per = prompt_part(p, x.keys), in = (int)blockIdx.y * RB + (int)threadIdx.x / TR, e = 4 * ((int)threadIdx.x % TR);
    const int row = kPrRows * x.tile + in;
    if (per >= x.keys || row >= x.n) return;              // one part, or no such tile or row
    const int parts = (x.keys + per - 1) / per;
    const int64_t at = ((int64_t)tile * p.Hq + head) * p.split * kPrRows + in;
    constexpr int G = 8;                       // parts read at a time
    float2 ml[kPrMaxSplit];
    float4 v[G];
#pragma unroll
    for (int i = 0; i < kPrMaxSplit; ++i) {
        ml[i] = float2{-INFINITY, 0.0f};
        if (i < parts) ml[i] = *reinterpret_cast<const float2 *>(p.ml + 2 * (at + (int64_t)i * kPrRows));
    }
    auto fetch = [&](int first) {
#pragma unroll
        for (int i = 0; i < G; ++i) {
            v[i] = float4{0.0f, 0.0f, 0.0f, 0.0f};
            if (first + i < parts) v[i] = *reinterpret_cast<const float4 *>(p.part + (at + (int64_t)(first + i) * kPrRows) * DV + e);
        }
    };
    fetch(0);
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPrMaxSplit; ++i) mx = fmaxf(mx, ml[i].x);
    const float use = mx == -INFINITY ? 0.0f : mx;
    float l = 0.0f;
    float4 o = float4{0.0f, 0.0f, 0.0f, 0.0f};
    auto add = [&](const float2 &s, const float4 &w) {
        const float f = s.x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(s.x - use);
        l += s.x == -INFINITY ? s.y : s.y * f;      // without a score above -inf: 0, or NaN
        o.x = fmaf(w.x, f, o.x), o.y = fmaf(w.y, f, o.y), o.z = fmaf(w.z, f, o.z), o.w = fmaf(w.w, f, o.w);
    };
#pragma unroll
    for (int i = 0; i < G; ++i) add(ml[i], v[i]);
    if (parts > G) {
        fetch(G);
#pragma unroll
        for (int i = 0; i < G; ++i) add(ml[G + i], v[i]);
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    *reinterpret_cast<uint2 *>(p.out + (int64_t)(x.q0 + row) * p.os + (int64_t)head * DV + e) =
        uint2{at_pack(o.x * inv, o.y * inv), at_pack(o.z * inv, o.w * inv)};
    if (p.lse && e == 0) p.lse[(int64_t)(x.q0 + row) * p.Hq + head] = l == 0.0f ? -INFINITY : (use + __log2f(l)) * kLn2;
}

template <int DK, int DV>
k3moe_status launch(const PromptParams &p, unsigned tiles, hipStream_t s)
{
    constexpr int lds = 2 * kAtKeys * (DK + DV) * 2;
    static std::atomic<uint64_t> allowed{0};
    if (!allow_lds(reinterpret_cast<const void *>(k_attention<DK, DV>), lds, allowed)) return K3MOE_E_HIP;
    k_attention<DK, DV><<<tiles * (unsigned)(p.Hq * p.split), 64 * kPrWaves, lds, s>>>(p);
    if (p.split > 1) k_attention_join<DV><<<dim3(tiles * (unsigned)p.Hq, kPrRows * DV / 1024), 256, 0, s>>>(p);
    return hipGetLastError() == hipSuccess ? K3MOE_OK : K3MOE_E_HIP;
}

// Tiles of queries at most: a sequence of n > 0 has (n + 127) / 128, rounded down.
int64_t prompt_tiles(int64_t seqs, int64_t Tq)
{
    const int64_t all = (Tq + (kPrRows - 1) * seqs) / kPrRows;
    return all < Tq ? all : Tq;
}

// Parts of a tile's keys. A tile of 64 keys costs a block 1.2 us (less where blocks share a CU), a part's writing and
// reading 1 / 50 us of the whole launch, the join's launch 4: of s parts of K tiles each over b blocks the time
// 1.2 K / s + b s / 50 + 4 is least at s * s = 60 K / b, and half of that fits the measurements where more than 256
// blocks share CUs. Queries x keys x heads of width 128, one part and what the rule takes: 1 x 512 x 8: 11.3 and
// 8.2 us, 64 x 4096 x 32: 71 and 23, 256 x 16384 x 8: 272 and 36, 1024 x 4096 x 32: 84 and 80. Where it takes one part:
// 1024 x 2048 x 32: 43, in three 58. Below 384 keys the parts do not pay for the join (1 x 256 x 8: 7.9 and 8.3, 320: 9.6
// and 10.0; 384: 9.8 and 8.3, 511: 13.5 and 10.0).
int prompt_split(int64_t seqs, int64_t Tq, int64_t Tk, int64_t Hq)
{
    if (seqs <= 0 || Tq <= 0) return 1;
    const int64_t blocks = prompt_tiles(seqs, Tq) * Hq, keys = Tk / seqs / kAtKeys;
    int s = 1;
    if (keys < kPrFrom) return s;
    for (int n = 2; n <= kPrMaxSplit && n * blocks <= kPrBlocks && n * kPrLeast <= keys; ++n)
        if (n * n * blocks <= kPrGain * keys * (n * blocks <= kPrBlocks / 2 ? 2 : 1)) s = n;
    return s;
}

// The same for every split, so that one workspace serves calls of all sizes.
size_t prompt_bytes(int64_t v_dim) { return (size_t)kPrBlocks * (kPrRows * (size_t)(v_dim + 2) * 4 + sizeof(int4)); }

bool at(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

}  // namespace
}  // namespace k3moe

using namespace k3moe;

extern "C" k3moe_status k3moe_attention(const uint16_t *q, int64_t q_stride, const uint16_t *k, int64_t k_stride,
                                        const uint16_t *v, int64_t v_stride, const int32_t *cu_q, const int32_t *cu_k,
                                        int32_t seqs, int32_t Tq, int32_t Tk, int32_t q_heads, int32_t kv_heads,
                                        int32_t k_dim, int32_t v_dim, float scale, int32_t causal, uint16_t *out,
                                        int64_t out_stride, float *lse, void *workspace, size_t workspace_bytes,
                                        void *stream)
{
    if (seqs < 0 || Tq < 0 || Tk < 0 || q_heads <= 0 || kv_heads <= 0 || q_heads % kv_heads || causal < 0 || causal > 1 ||
        !(scale > 0.0f && scale <= 0x1p64f))
        return K3MOE_E_INVALID_ARG;
    if (!((k_dim == v_dim && (k_dim == 64 || k_dim == 128)) || (k_dim == 192 && v_dim == 128)))
        return K3MOE_E_UNSUPPORTED_SHAPE;
    if (seqs == 0 || Tq == 0) return K3MOE_OK;
    if (!q || !cu_q || !out || (Tk > 0 && (!k || !v))) return K3MOE_E_INVALID_ARG;
    const int64_t qw = (int64_t)q_heads * k_dim, kw = (int64_t)kv_heads * k_dim, vw = (int64_t)kv_heads * v_dim,
                  ow = (int64_t)q_heads * v_dim;
    if (Tq == 1) q_stride = qw, out_stride = ow;
    if (Tk <= 1) k_stride = kw, v_stride = vw;
    if (q_stride < qw || k_stride < kw || v_stride < vw || out_stride < ow) return K3MOE_E_INVALID_ARG;
    constexpr int64_t kMaxStride = 1 << 24;
    if (q_stride > kMaxStride || k_stride > kMaxStride || v_stride > kMaxStride || out_stride > kMaxStride)
        return K3MOE_E_UNSUPPORTED_SHAPE;
    if (!at(q, 16) || !at(k, 16) || !at(v, 16) || !at(out, 16) || q_stride % 8 || k_stride % 8 || v_stride % 8 || out_stride % 8 ||
        !at(cu_q, 4) || !at(cu_k, 4) || !at(lse, 4))
        return K3MOE_E_ALIGNMENT;
    const int64_t tiles = prompt_tiles(seqs, Tq);
    if (tiles * q_heads >= (int64_t)1 << 24 || seqs > 1 << 30) return K3MOE_E_UNSUPPORTED_SHAPE;   // work-items are counted in 32 bits
    const int split = workspace ? prompt_split(seqs, Tq, Tk, q_heads) : 1;
    if (workspace && (!at(workspace, 256) || (split > 1 && workspace_bytes < prompt_bytes(v_dim)))) return K3MOE_E_WORKSPACE;
    PromptParams p{};
    p.q = q, p.k = k, p.v = v, p.cu_q = cu_q, p.cu_k = cu_k, p.out = out, p.lse = lse;
    p.qs = q_stride, p.ks = k_stride, p.vs = v_stride, p.os = out_stride;
    p.seqs = seqs, p.Tq = Tq, p.Tk = Tk, p.Hq = q_heads, p.group = q_heads / kv_heads, p.causal = causal, p.scale = scale;
    p.split = split;
    if (p.split > 1) {
        p.joins = static_cast<int4 *>(workspace);
        p.part = reinterpret_cast<float *>(p.joins + kPrBlocks);
        p.ml = p.part + (size_t)(tiles * q_heads * p.split) * kPrRows * (size_t)v_dim;
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    const unsigned t = (unsigned)tiles;
    return k_dim == 64 ? launch<64, 64>(p, t, s) : k_dim == 128 ? launch<128, 128>(p, t, s) : launch<192, 128>(p, t, s);
}

extern "C" k3moe_status k3moe_attention_workspace_size(int32_t seqs, int32_t Tq, int32_t Tk, int32_t q_heads, int32_t v_dim,
                                                       size_t *bytes)
{
    if (!bytes || seqs < 0 || Tq < 0 || Tk < 0 || q_heads <= 0) return K3MOE_E_INVALID_ARG;
    if (v_dim != 64 && v_dim != 128) return K3MOE_E_UNSUPPORTED_SHAPE;
    // one query over all keys is split if any call of up to these sizes is: fewer blocks and longer sequences split first
    *bytes = prompt_split(seqs < 1 ? seqs : 1, Tq < 1 ? Tq : 1, Tk, q_heads) < 2 ? 0 : prompt_bytes(v_dim);
    return K3MOE_OK;
}
