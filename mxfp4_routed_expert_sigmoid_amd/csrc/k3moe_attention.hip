// Attention of packed sequences (k3moe_attention): per sequence, query head and
// query i of n over keys j of N
//   s_j = scale q_i . k_j,  out = sum_j e^(s_j) v_j / sum_j e^(s_j),
//   lse = log sum_j e^(s_j),  causal: j <= i + N - n
// in one pass over the keys with the running maximum and sum.
//
// A block of four waves owns 128 queries of one head, a wave 32 of them
// (k3moe_attn.h). Tiles of 64 keys and values go through LDS by direct loads
// into two buffers, one barrier per tile.
#include "k3moe_attn.h"

namespace k3moe {
namespace {

constexpr int kPrWaves = 4, kPrRows = kPrWaves * kAtRows;
constexpr unsigned kPrCus = 256;

struct PromptParams {
    const uint16_t *q, *k, *v;
    const int32_t *cu_q, *cu_k;
    uint16_t *out;
    float *lse;
    int64_t qs, ks, vs, os;   // row strides, elements
    int seqs, Tq, Tk, Hq, group, causal;
    float scale;
};

// SPLIT: four more waves take the second half of the keys, with buffers of their own.
template <int DK, int DV, bool SPLIT>
__global__ __launch_bounds__(64 * kPrWaves * (SPLIT ? 2 : 1), 2) void k_attention(PromptParams p)
{
#ifdef __HIP_DEVICE_COMPILE__
    constexpr int KB = kAtKeys * DK * 2, VB = kAtKeys * DV * 2;
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, h = lane >> 5, l32 = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % kPrWaves;
    const int part = SPLIT ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / kPrWaves : 0;
    const int head = blockIdx.x % p.Hq;
    int tile = blockIdx.x / p.Hq;

    // This block's sequence and tile within it: 64 sequences at a time.
    int b = -1, q0 = 0, n = 0;
    for (int b0 = 0; b0 < p.seqs && b < 0; b0 += 64) {
        int lo = 0, hi = 0;
        if (b0 + lane < p.seqs) {
            lo = min(max(p.cu_q[b0 + lane], 0), p.Tq);
            hi = min(max(p.cu_q[b0 + lane + 1], lo), p.Tq);
        }
        const int mine = (hi - lo + kPrRows - 1) / kPrRows;
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int x = __shfl_up(upto, o);
            if (lane >= o) upto += x;
        }
        const uint64_t past = __ballot(upto > tile);
        if (past) {
            const int at = __builtin_ctzll(past);
            b = b0 + at;
            q0 = __builtin_amdgcn_readlane(lo, at);
            n = __builtin_amdgcn_readlane(hi, at) - q0;
            tile = __builtin_amdgcn_readlane(upto, at) - 1 - tile;   // the longest first
        } else {
            tile -= __builtin_amdgcn_readlane(upto, 63);
        }
    }
    if (b < 0) return;
    const int32_t *cu = p.cu_k ? p.cu_k : p.cu_q;
    const int k0 = min(max(cu[b], 0), p.Tk), N = min(max(cu[b + 1], k0), p.Tk) - k0;

    const int row = kPrRows * tile + kAtRows * wave + l32;   // this lane's query of the sequence
    const bool have = row < n;
    AttRows<DK, DV> r;
    {
        const uint16_t *qp = p.q + (int64_t)(q0 + min(row, n - 1)) * p.qs + (int64_t)head * DK + 8 * h;
#pragma unroll
        for (int k = 0; k < DK / 16; ++k) r.q[k] = as_bf8(*reinterpret_cast<const u4 *>(qp + 16 * k));
    }
    r.clear();
    // keys this lane's row, this wave's and this block's last row see: the first `see` ones
    const int see = p.causal ? min(row + 1 + N - n, N) : N;
    const int wfirst = kPrRows * tile + kAtRows * wave, wlast = min(wfirst + kAtRows, n) - 1;
    const int wsee = wfirst >= n ? 0 : p.causal ? wlast + 1 + N - n : N;
    const int wall = wfirst >= n ? 0 : p.causal ? wfirst + 1 + N - n : N;      // every row of the wave sees these
    const int bsee = p.causal ? min(kPrRows * (tile + 1), n) + N - n : N;
    const int all = (max(bsee, 0) + kAtKeys - 1) / kAtKeys, steps = SPLIT ? (all + 1) / 2 : all;
    const int t0 = part * steps, t1 = min(t0 + steps, all);                    // this part's tiles

    const int kvh = head / p.group;
    const uint16_t *kp = p.k + (int64_t)k0 * p.ks + (int64_t)kvh * DK, *vp = p.v + (int64_t)k0 * p.vs + (int64_t)kvh * DV;
    // Keys run a tile ahead of the values: tile t's scores are computed beside the weights of tile t - 1. i counts a
    // part's tiles.
    const uint8_t *buf = lds + part * 2 * (KB + VB);
    RowStage<DK, true> sk;
    RowStage<DV, false> sv;
    sk.init(p.ks), sv.init(p.vs);
    auto ktile = [&](int i) { return buf + (i & 1) * KB; };
    auto vtile = [&](int i) { return buf + 2 * KB + (i & 1) * VB; };
    // a wave loads 16 of a tile's rows; those behind the last key read as zeros
    auto load_k = [&](int i) {
        const int at = (t0 + i) * kAtKeys + 16 * wave;
        if (t0 + i < t1) sk.load(kp + (int64_t)at * p.ks, p.ks, N - at, ktile(i) + 16 * wave * DK * 2);
    };
    auto load_v = [&](int i) {
        const int at = (t0 + i) * kAtKeys + 16 * wave;
        if (t0 + i < t1) sv.load(vp + (int64_t)at * p.vs, p.vs, N - at, vtile(i) + 16 * wave * DV * 2);
    };
    const float c = p.scale * kLog2e;
    if (steps > 0) {
        load_k(0), load_k(1), load_v(0);
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
            att_tile(r, s, mx, o, buf + KB, vtile(0), c);
            at_barrier();
            load_k(i + 3), load_v(i + 2);
            att_tile(r, o, mx, s, buf, vtile(1), c);
        }
        for (; i < steps; ++i) {
            at_barrier();
            load_k(i + 2), load_v(i + 1);
            const int first = (t0 + i) * kAtKeys;
            if (t0 + i < t1 && first < wsee) att_tile_masked(r, s, ktile(i + 1), vtile(i), c, low_bits(see - first));
        }
    }

    float l = r.l + __shfl_xor(r.l, 32);
    if constexpr (SPLIT) {
        // the second half's rows join the first's through LDS, in the lanes' own order
        at_barrier();
        float *x = reinterpret_cast<float *>(lds) + wave * 64 * (16 * (DV / 32) + 2) + lane;
        if (part == 1) {
            x[0] = r.m, x[64] = l;
#pragma unroll
            for (int d = 0; d < DV / 32; ++d)
#pragma unroll
                for (int e = 0; e < 16; ++e) x[64 * (2 + 16 * d + e)] = r.o[d][e];
        }
        at_barrier();
        if (part == 1) return;
        const float m1 = x[0], mn = fmaxf(r.m, m1);
        const float f0 = r.m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((r.m - mn) * c);
        const float f1 = m1 == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((m1 - mn) * c);
        // (a part whose scores were all -inf has neither sum nor values; one with NaN has, whatever its maximum)
        l = (r.m == -INFINITY ? l : l * f0) + (m1 == -INFINITY ? x[64] : x[64] * f1);
        r.m = mn;
#pragma unroll
        for (int d = 0; d < DV / 32; ++d)
#pragma unroll
            for (int e = 0; e < 16; ++e) r.o[d][e] = r.o[d][e] * f0 + x[64 * (2 + 16 * d + e)] * f1;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    if (!have) return;
    if (p.lse && h == 0)
        p.lse[(int64_t)(q0 + row) * p.Hq + head] = l == 0.0f ? -INFINITY : fmaf(r.m, c, __log2f(l)) * kLn2;
    uint16_t *op = p.out + (int64_t)(q0 + row) * p.os + (int64_t)head * DV + 4 * h;
#pragma unroll
    for (int d = 0; d < DV / 32; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<uint2 *>(op + 32 * d + 2 * i) = uint2{
                at_bf16(r.o[d][i] * inv) | (at_bf16(r.o[d][i + 1] * inv) << 16),
                at_bf16(r.o[d][i + 2] * inv) | (at_bf16(r.o[d][i + 3] * inv) << 16)};
#endif
}

template <int DK, int DV, bool SPLIT>
k3moe_status launch(const PromptParams &p, unsigned grid, hipStream_t s)
{
    constexpr int lds = 2 * kAtKeys * (DK + DV) * 2 * (SPLIT ? 2 : 1);
    static_assert(!SPLIT || lds >= kPrWaves * 64 * (DV / 2 + 2) * 4, "the halves' join fits the tiles");
    static const hipError_t allowed =
        hipFuncSetAttribute(reinterpret_cast<const void *>(k_attention<DK, DV, SPLIT>), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (allowed != hipSuccess) return K3MOE_E_HIP;
    k_attention<DK, DV, SPLIT><<<grid, 64 * kPrWaves * (SPLIT ? 2 : 1), lds, s>>>(p);
    return hipGetLastError() == hipSuccess ? K3MOE_OK : K3MOE_E_HIP;
}

template <int DK, int DV>
k3moe_status launch(const PromptParams &p, unsigned grid, hipStream_t s)
{
    // no more tiles than CUs: a CU takes the waves of two blocks, so a tile gets them all
    return grid <= kPrCus ? launch<DK, DV, true>(p, grid, s) : launch<DK, DV, false>(p, grid, s);
}

bool at(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

}  // namespace
}  // namespace k3moe

using namespace k3moe;

extern "C" k3moe_status k3moe_attention(const uint16_t *q, int64_t q_stride, const uint16_t *k, int64_t k_stride,
                                        const uint16_t *v, int64_t v_stride, const int32_t *cu_q, const int32_t *cu_k,
                                        int32_t seqs, int32_t Tq, int32_t Tk, int32_t q_heads, int32_t kv_heads,
                                        int32_t k_dim, int32_t v_dim, float scale, int32_t causal, uint16_t *out,
                                        int64_t out_stride, float *lse, void *stream)
{
    if (seqs < 0 || Tq < 0 || Tk < 0 || q_heads <= 0 || kv_heads <= 0 || q_heads % kv_heads || causal < 0 || causal > 1 ||
        !(scale > 0.0f && scale < INFINITY))
        return K3MOE_E_INVALID_ARG;
    if (!((k_dim == v_dim && (k_dim == 64 || k_dim == 128)) || (k_dim == 192 && v_dim == 128))) return K3MOE_E_UNSUPPORTED_SHAPE;
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
    // a sequence has at most one tile that is not full
    int64_t tiles = (int64_t)Tq / kPrRows + seqs;
    if (tiles > Tq) tiles = Tq;
    if (tiles * q_heads >= (int64_t)1 << 24) return K3MOE_E_UNSUPPORTED_SHAPE;   // work-items are counted in 32 bits
    PromptParams p{};
    p.q = q, p.k = k, p.v = v, p.cu_q = cu_q, p.cu_k = cu_k, p.out = out, p.lse = lse;
    p.qs = q_stride, p.ks = k_stride, p.vs = v_stride, p.os = out_stride;
    p.seqs = seqs, p.Tq = Tq, p.Tk = Tk, p.Hq = q_heads, p.group = q_heads / kv_heads, p.causal = causal, p.scale = scale;
    const unsigned grid = (unsigned)(tiles * q_heads);
    hipStream_t s = static_cast<hipStream_t>(stream);
    return k_dim == 64 ? launch<64, 64>(p, grid, s) : k_dim == 128 ? launch<128, 128>(p, grid, s) : launch<192, 128>(p, grid, s);
}
