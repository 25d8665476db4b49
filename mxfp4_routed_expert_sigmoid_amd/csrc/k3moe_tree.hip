// Attention of drafted tokens over the paged cache (k3moe_tree_attention): per
// sequence, drafted token i and query head
//   out = sum_j e^(s_j) v_j / sum_j e^(s_j),  s_j = scale q_i . k_j,
// over the context and the drafted tokens whose bits are set in i's word.
//
// The rows that share a key/value head, (token, head of the group), are one
// matrix: 128 of them per block. The work is a line of units, a unit being 64
// keys of one (sequence, key/value head, 128 rows), cut into equal runs, one
// per block, so that sequences of any lengths fill the card alike. What a run
// holds whole is written at once; cut ends (two per block at most) go to the
// workspace as unnormalised sums with their maximum, and a second kernel joins
// them in their order.
#include "k3moe_attn.h"

namespace k3moe {
namespace {

constexpr int kTrWaves = 4, kTrRows = kTrWaves * kAtRows;
constexpr int kTrBlocks = 512;   // runs: two blocks of 80 KB of LDS or less per CU
constexpr int kTrLeast = 2;      // units of a run at least
constexpr int kTrMaxDraft = 64;  // bits of a word

struct TreeParams {
    const uint16_t *q;
    const uint8_t *kc, *vc, *ks, *vs;
    const int32_t *pages, *lens, *cu;
    const uint64_t *tree;
    uint16_t *out;
    float *lse, *part, *ml;   // part [2 kTrBlocks][rows][DV], ml [2 kTrBlocks][rows][2]
    int64_t qs, os;
    int seqs, Tq, maxq, Hq, Hkv, group, n_pages, lpage, width;
    float scale;
};

// What a sequence has to do.
struct TreeSeq {
    int q0, n, ctx, keys, kt, rt;   // first row, drafted tokens, context, keys, tiles of keys and of rows
    int64_t units;
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeParams &p, int b)
{
    TreeSeq s{};
    if (b >= p.seqs) return s;
    int hi;
    if (p.cu) {
        s.q0 = min(max(p.cu[b], 0), p.Tq);
        hi = min(max(p.cu[b + 1], s.q0), p.Tq);
    } else {
        const int each = p.Tq / p.seqs;
        s.q0 = b * each, hi = s.q0 + each;
    }
    s.n = min(hi - s.q0, p.maxq);
    s.ctx = max(p.lens[b], 0);
    s.keys = (int)min((int64_t)s.ctx + s.n, (int64_t)p.width << p.lpage);
    s.kt = max(1, (s.keys + kAtKeys - 1) / kAtKeys);   // a row without a key is written too
    s.rt = (s.n * p.group + kTrRows - 1) / kTrRows;
    s.units = (int64_t)p.Hkv * s.rt * s.kt;
    return s;
}

__device__ __forceinline__ int64_t shfl_up64(int64_t v, int o)
{
    const uint32_t lo = __shfl_up((uint32_t)v, o), hi = __shfl_up((uint32_t)(v >> 32), o);
    return (int64_t)(((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ int64_t lane64(int64_t v, int l)
{
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, l);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), l);
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

// Units of the sequences b0 .. b0 + 63 up to and with this lane's.
__device__ __forceinline__ int64_t tree_scan(const TreeSeq &s)
{
    const int lane = threadIdx.x & 63;
    int64_t upto = s.units;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int64_t x = shfl_up64(upto, o);
        if (lane >= o) upto += x;
    }
    return upto;
}

__device__ __forceinline__ int64_t run_length(int64_t units)
{
    const int64_t r = (units + kTrBlocks - 1) / kTrBlocks;
    return r < kTrLeast ? kTrLeast : r;
}

// The sum over all sequences, and (find >= 0) the sequence that holds unit `find` with the units in front of it.
__device__ __forceinline__ int64_t tree_total(const TreeParams &p)
{
    const int lane = threadIdx.x & 63;
    int64_t total = 0;
    for (int b0 = 0; b0 < p.seqs; b0 += 64) total += lane64(tree_scan(tree_seq(p, b0 + lane)), 63);
    return total;
}
__device__ __forceinline__ int tree_find(const TreeParams &p, int64_t unit, int64_t &front)
{
    const int lane = threadIdx.x & 63;
    front = 0;
    for (int b0 = 0; b0 < p.seqs; b0 += 64) {
        const TreeSeq s = tree_seq(p, b0 + lane);
        const int64_t upto = tree_scan(s) + front;
        const uint64_t past = __ballot(upto > unit);
        if (past) {
            const int at = __builtin_ctzll(past);
            front = lane64(upto - s.units, at);
            return b0 + at;
        }
        front = lane64(upto, 63);
    }
    return -1;
}

#ifdef __HIP_DEVICE_COMPILE__
typedef __attribute__((address_space(3))) void lds_void;

__device__ __forceinline__ u4 expand_pair(uint32_t lo, uint32_t hi, float f)
{
    const bf2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, f, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, f, true);
    const bf2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, f, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, f, true);
    const bf8 v = bf8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    u4 r;
    __builtin_memcpy(&r, &v, 16);
    return r;
}

// One side (keys or values) of the cache: a wave stages its 16 rows of a tile, all in one page.
template <int D, bool X8>
struct PageStage {
    u4 w[X8 ? D / 64 : 1];
    uint32_t sc[X8 ? D / 64 : 1];

    // base: the head's rows of the page from this wave's first on; rows: how many of the 16 exist
    template <class Slot>
    __device__ __forceinline__ void issue(const uint8_t *base, const uint8_t *sbase, int rows, const uint8_t *lds, Slot slot)
    {
        const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(base), 0, kAtOut, 0x00020000);
        if constexpr (!X8) {
            constexpr int SL = D / 8, N = 16 * SL / 64;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int at = (wave * N + i) * 64 + lane, row = at / SL, s = slot(row, at % SL) - row * SL, r16 = row - 16 * wave;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)(lds + (wave * N + i) * 1024), 16,
                                                         (int)(r16 < rows ? (uint32_t)(r16 * D * 2 + 16 * s) : kAtOut), 0, 0, 0);
            }
        } else {
            const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(sbase), 0, kAtOut, 0x00020000);
            typedef unsigned u4v __attribute__((ext_vector_type(4)));
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const int at = 64 * i + lane, row = at / (D / 16), sub = at % (D / 16);
                const u4v x = __builtin_amdgcn_raw_buffer_load_b128(r, (int)(row < rows ? (uint32_t)(16 * at) : kAtOut), 0, 0);
                w[i] = u4{x[0], x[1], x[2], x[3]};
                sc[i] = __builtin_amdgcn_raw_buffer_load_b8(rs, (int)(row < rows ? (uint32_t)(row * (D / 32) + sub / 2) : kAtOut), 0, 0);
            }
        }
    }
    template <class Slot>
    __device__ __forceinline__ void commit(uint8_t *lds, Slot slot)
    {
        if constexpr (X8) {
            const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const int at = 64 * i + lane, row = 16 * wave + at / (D / 16), sub = at % (D / 16);
                const bool drop = sc[i] == 255u;   // such a group is zero, whatever its codes
                const float f = e8m0_to_f32(sc[i]);
                const u4 x = drop ? u4{0u, 0u, 0u, 0u} : w[i];
                *reinterpret_cast<u4 *>(lds + 16 * slot(row, 2 * sub)) = expand_pair(x.x, x.y, f);
                *reinterpret_cast<u4 *>(lds + 16 * slot(row, 2 * sub + 1)) = expand_pair(x.z, x.w, f);
            }
        }
    }
};
#endif

template <int DK, int DV, bool X8>
__global__ __launch_bounds__(64 * kTrWaves, 2) void k_tree(TreeParams p)
{
#ifdef __HIP_DEVICE_COMPILE__
    constexpr int KB = kAtKeys * DK * 2, VB = kAtKeys * DV * 2, EB = X8 ? 1 : 2;
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5, l32 = lane & 31;
    const int64_t total = tree_total(p), per = run_length(total);
    int64_t u = per * blockIdx.x;
    const int64_t end = min(u + per, total);
    if (u >= end) return;
    int64_t front;
    int b = tree_find(p, u, front);
    TreeSeq s = tree_seq(p, b);
    const int page = 1 << p.lpage;
    const float c = p.scale * kLog2e;

    while (true) {
        // the segment that holds unit u: tiles t0 .. t1 of (b, kvh, rows)
        const int64_t in = u - front;
        const int seg = (int)(in / s.kt), t0 = (int)(in - (int64_t)seg * s.kt);
        const int kvh = seg / s.rt, rows0 = (seg - kvh * s.rt) * kTrRows;
        const int t1 = (int)min((int64_t)s.kt, t0 + (end - u));

        const int m = rows0 + kAtRows * wave + l32;                 // (token, head of the group)
        const int i = min(m / p.group, s.n - 1), head = kvh * p.group + m % p.group;
        const bool have = m < s.n * p.group, busy = rows0 + kAtRows * wave < s.n * p.group;
        const uint64_t word = (p.tree ? p.tree[s.q0 + i] : low_bits(i + 1)) & low_bits(s.n);
        AttRows<DK, DV> r;
        {
            const uint16_t *qp = p.q + (int64_t)(s.q0 + i) * p.qs + (int64_t)head * DK + 8 * h;
#pragma unroll
            for (int k = 0; k < DK / 16; ++k) r.q[k] = as_bf8(*reinterpret_cast<const u4 *>(qp + 16 * k));
        }
        r.clear();

        // page numbers of a tile's four runs of 16 keys, and which of them are in the cache
        const int32_t *table = p.pages + (int64_t)b * p.width;
        auto lookup = [&](int t, int &own) {   // own: the page of this wave's rows, -1: none
            uint32_t ok = 0;
            own = -1;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int pos = t * kAtKeys + 16 * g;
                const int id = pos < s.keys ? __builtin_amdgcn_readfirstlane(table[pos >> p.lpage]) : -1;
                const bool in_cache = id >= 0 && id < p.n_pages;
                ok |= in_cache ? 1u << g : 0u;
                if (g == wave) own = in_cache ? id : -1;
            }
            return ok;
        };
        PageStage<DK, X8> sk;
        PageStage<DV, X8> sv;
        // Keys run a tile ahead of the values: tile t's scores are there before its weights are taken. What goes through
        // registers (8-bit pages) is written behind the tile's work, before the barrier in front of its use.
        auto where = [&](int t, int own, int &rows) {
            const int pos = t * kAtKeys + 16 * wave;
            rows = own < 0 ? 0 : min(s.keys - pos, 16);
            return ((int64_t)max(own, 0) * p.Hkv + kvh) * page + (pos & (page - 1));
        };
        auto issue_k = [&](int t, int own) {
            int rows;
            const int64_t row = where(t, own, rows);
            sk.issue(p.kc + row * DK * EB, X8 ? p.ks + row * (DK / 32) : nullptr, rows, lds + ((t - t0) & 1) * KB, k_slot<DK>);
        };
        auto issue_v = [&](int t, int own) {
            int rows;
            const int64_t row = where(t, own, rows);
            sv.issue(p.vc + row * DV * EB, X8 ? p.vs + row * (DV / 32) : nullptr, rows, lds + 2 * KB + ((t - t0) & 1) * VB, v_slot<DV>);
        };
        auto commit_k = [&](int t) { sk.commit(lds + ((t - t0) & 1) * KB, k_slot<DK>); };
        auto commit_v = [&](int t) { sv.commit(lds + 2 * KB + ((t - t0) & 1) * VB, v_slot<DV>); };

        at_barrier();       // the last segment's tiles are read
        int own0, own1 = -1, own2 = -1;            // this wave's pages of tiles t, t + 1, t + 2
        uint32_t ok = lookup(t0, own0), ok1 = 0;
        if (t0 + 1 < t1) ok1 = lookup(t0 + 1, own1);
        issue_k(t0, own0), issue_v(t0, own0);
        commit_k(t0), commit_v(t0);
        if (t0 + 1 < t1) issue_k(t0 + 1, own1), commit_k(t0 + 1);
        at_barrier();
        v16f sc[2];
        if (busy) att_scores(sc, r, lds);
        for (int t = t0; t < t1; ++t) {
            const int first = t * kAtKeys;
            uint32_t ok2 = 0;
            at_barrier();
            if (t + 2 < t1) ok2 = lookup(t + 2, own2), issue_k(t + 2, own2);
            if (t + 1 < t1) issue_v(t + 1, own1);
            if (busy) {
                const uint8_t *nk = lds + ((t + 1 - t0) & 1) * KB, *vt = lds + 2 * KB + ((t - t0) & 1) * VB;
                const int a = s.ctx - first;   // the tile's keys in front of the drafted ones
                uint64_t seen = low_bits(a) | (a >= 64 || a <= -64 ? 0ull : a >= 0 ? word << a : word >> -a);
                seen &= low_bits(s.keys - first);
#pragma unroll
                for (int g = 0; g < 4; ++g) seen &= ok >> g & 1 ? ~0ull : ~(0xffffull << (16 * g));
                att_tile_masked(r, sc, nk, vt, c, seen);
            }
            if (t + 2 < t1) commit_k(t + 2);
            if (t + 1 < t1) commit_v(t + 1);
            ok = ok1, ok1 = ok2, own1 = own2;
        }

        const float l = r.l + __shfl_xor(r.l, 32);
        if (t0 == 0 && t1 == s.kt) {
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            if (have) {
                if (p.lse && h == 0)
                    p.lse[(int64_t)(s.q0 + i) * p.Hq + head] = l == 0.0f ? -INFINITY : fmaf(r.m, c, __log2f(l)) * kLn2;
                uint16_t *op = p.out + (int64_t)(s.q0 + i) * p.os + (int64_t)head * DV + 4 * h;
#pragma unroll
                for (int d = 0; d < DV / 32; ++d)
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        *reinterpret_cast<uint2 *>(op + 32 * d + 2 * e) = uint2{
                            at_bf16(r.o[d][e] * inv) | (at_bf16(r.o[d][e + 1] * inv) << 16),
                            at_bf16(r.o[d][e + 2] * inv) | (at_bf16(r.o[d][e + 3] * inv) << 16)};
            }
        } else if (have) {
            // a run cut in front goes to the block's first place, one cut behind only to its second
            const int64_t at = (int64_t)(2 * blockIdx.x + (t0 == 0)) * kTrRows + (m - rows0);
            float *op = p.part + at * DV + 4 * h;
#pragma unroll
            for (int d = 0; d < DV / 32; ++d)
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    *reinterpret_cast<float4 *>(op + 32 * d + 2 * e) = float4{r.o[d][e], r.o[d][e + 1], r.o[d][e + 2], r.o[d][e + 3]};
            if (h == 0) *reinterpret_cast<float2 *>(p.ml + 2 * at) = float2{r.m * c, l};   // c > 0: -inf stays
        }

        u += t1 - t0;
        if (u >= end) return;
        while (u >= front + s.units) {
            front += s.units;
            s = tree_seq(p, ++b);
        }
    }
#endif
}

// Joins the cut ends: one wave per (drafted token, head).
template <int DV>
__global__ __launch_bounds__(256) void k_tree_join(TreeParams p)
{
    const int lane = threadIdx.x & 63;
    const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (item >= (int64_t)p.Tq * p.Hq) return;
    const int t = (int)(item / p.Hq), head = (int)(item % p.Hq);

    int64_t total = 0, front = -1;
    TreeSeq s{};
    for (int b0 = 0; b0 < p.seqs; b0 += 64) {
        const TreeSeq x = tree_seq(p, b0 + lane);
        const int64_t upto = tree_scan(x) + total;
        const uint64_t mine = __ballot(t >= x.q0 && t < x.q0 + x.n);
        if (mine && front < 0) {
            const int at = __builtin_ctzll(mine);
            front = lane64(upto - x.units, at);
            s = tree_seq(p, b0 + at);
        }
        total = lane64(upto, 63);
    }
    if (front < 0) return;   // a row of no sequence
    const int64_t per = run_length(total);
    const int m = (t - s.q0) * p.group + head % p.group, rt = m / kTrRows;
    const int64_t u0 = front + ((int64_t)(head / p.group) * s.rt + rt) * s.kt, u1 = u0 + s.kt;
    const int w0 = (int)(u0 / per), w1 = (int)((u1 - 1) / per);
    if (w0 == w1) return;    // written whole
    auto place = [&](int w) { return ((int64_t)(2 * w + (w == w0)) * kTrRows + (m - rt * kTrRows)); };
    // 64 runs at a time: their maxima and sums, then their sums of values
    float mx = -INFINITY;
    for (int w = w0 + lane; w <= w1; w += 64) mx = fmaxf(mx, p.ml[2 * place(w)]);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
    const float use = mx == -INFINITY ? 0.0f : mx;
    float l = 0.0f, o0 = 0.0f, o1 = 0.0f;
    for (int w = w0; w <= w1; ++w) {
        const int64_t at = place(w);
        const float f = __builtin_amdgcn_exp2f(p.ml[2 * at] - use);
        l = fmaf(p.ml[2 * at + 1], f, l);
        o0 = fmaf(p.part[at * DV + lane], f, o0);
        if constexpr (DV == 128) o1 = fmaf(p.part[at * DV + 64 + lane], f, o1);
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t *op = p.out + (int64_t)t * p.os + (int64_t)head * DV;
    op[lane] = (uint16_t)at_bf16(o0 * inv);
    if constexpr (DV == 128) op[64 + lane] = (uint16_t)at_bf16(o1 * inv);
    if (p.lse && lane == 0) p.lse[(int64_t)t * p.Hq + head] = l == 0.0f ? -INFINITY : (use + __log2f(l)) * kLn2;
}

template <int DK, int DV, bool X8>
k3moe_status launch(const TreeParams &p, hipStream_t s)
{
    constexpr int lds = 2 * kAtKeys * (DK + DV) * 2;
    static const hipError_t allowed =
        hipFuncSetAttribute(reinterpret_cast<const void *>(k_tree<DK, DV, X8>), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (allowed != hipSuccess) return K3MOE_E_HIP;
    k_tree<DK, DV, X8><<<kTrBlocks, 64 * kTrWaves, lds, s>>>(p);
    k_tree_join<DV><<<(unsigned)(((int64_t)p.Tq * p.Hq + 3) / 4), 256, 0, s>>>(p);
    return hipGetLastError() == hipSuccess ? K3MOE_OK : K3MOE_E_HIP;
}

bool at(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

size_t ws_bytes(int v_dim) { return (size_t)2 * kTrBlocks * kTrRows * (size_t)(v_dim + 2) * 4; }

}  // namespace
}  // namespace k3moe

using namespace k3moe;

extern "C" k3moe_status k3moe_tree_attention_workspace_size(int32_t q_heads, int32_t kv_heads, int32_t v_dim, int32_t max_q,
                                                            size_t *bytes)
{
    if (!bytes || q_heads <= 0 || kv_heads <= 0 || q_heads % kv_heads || max_q < 1) return K3MOE_E_INVALID_ARG;
    if ((v_dim != 64 && v_dim != 128) || max_q > kTrMaxDraft || q_heads > 4096) return K3MOE_E_UNSUPPORTED_SHAPE;
    *bytes = ws_bytes(v_dim);
    return K3MOE_OK;
}

extern "C" k3moe_status k3moe_tree_attention(const uint16_t *q, int64_t q_stride, const k3moe_pages *cache, const int32_t *pages,
                                             int32_t pages_width, const int32_t *lens, const int32_t *cu_q,
                                             const uint64_t *tree, int32_t seqs, int32_t Tq, int32_t max_q, int32_t q_heads,
                                             int32_t kv_heads, int32_t k_dim, int32_t v_dim, float scale, uint16_t *out,
                                             int64_t out_stride, float *lse, void *workspace, size_t workspace_bytes,
                                             void *stream)
{
    if (!cache || seqs < 0 || Tq < 0 || max_q < 1 || q_heads <= 0 || kv_heads <= 0 || q_heads % kv_heads || pages_width < 0 ||
        cache->pages < 0 || cache->page <= 0 || !(scale > 0.0f && scale < INFINITY))
        return K3MOE_E_INVALID_ARG;
    const int page = cache->page;
    if (!((k_dim == v_dim && (k_dim == 64 || k_dim == 128)) || (k_dim == 192 && v_dim == 128)) || max_q > kTrMaxDraft ||
        q_heads > 4096 || page < 16 || page > 1 << 20 || (page & (page - 1)) || (int64_t)pages_width * page > (int64_t)1 << 30)
        return K3MOE_E_UNSUPPORTED_SHAPE;
    if (seqs == 0 || Tq == 0) return K3MOE_OK;
    if (!cu_q && (Tq % seqs || Tq / seqs > max_q)) return K3MOE_E_INVALID_ARG;
    const bool x8 = cache->ks != nullptr;
    if (!q || !lens || !out || (pages_width > 0 && !pages) || (cache->vs != nullptr) != x8 ||
        (cache->pages > 0 && (!cache->k || !cache->v)))
        return K3MOE_E_INVALID_ARG;
    const int64_t qw = (int64_t)q_heads * k_dim, ow = (int64_t)q_heads * v_dim;
    if (Tq == 1) q_stride = qw, out_stride = ow;
    if (q_stride < qw || out_stride < ow) return K3MOE_E_INVALID_ARG;
    if (((int64_t)Tq * q_heads + 3) / 4 >= (int64_t)1 << 24) return K3MOE_E_UNSUPPORTED_SHAPE;   // work-items are counted in 32 bits
    if (!at(q, 16) || !at(out, 16) || q_stride % 8 || out_stride % 8 || !at(cache->k, 16) || !at(cache->v, 16) || !at(pages, 4) ||
        !at(lens, 4) || !at(cu_q, 4) || !at(tree, 8) || !at(lse, 4))
        return K3MOE_E_ALIGNMENT;
    if (!workspace || !at(workspace, 256) || workspace_bytes < ws_bytes(v_dim)) return K3MOE_E_WORKSPACE;
    TreeParams p{};
    p.q = q, p.kc = static_cast<const uint8_t *>(cache->k), p.vc = static_cast<const uint8_t *>(cache->v);
    p.ks = cache->ks, p.vs = cache->vs, p.pages = pages, p.lens = lens, p.cu = cu_q, p.tree = tree, p.out = out, p.lse = lse;
    p.part = static_cast<float *>(workspace);
    p.ml = p.part + (size_t)2 * kTrBlocks * kTrRows * (size_t)v_dim;
    p.qs = q_stride, p.os = out_stride, p.seqs = seqs, p.Tq = Tq, p.maxq = max_q, p.Hq = q_heads, p.Hkv = kv_heads;
    p.group = q_heads / kv_heads, p.n_pages = cache->pages, p.lpage = __builtin_ctz((unsigned)page), p.width = pages_width;
    p.scale = scale;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (k_dim == 64) return x8 ? launch<64, 64, true>(p, s) : launch<64, 64, false>(p, s);
    if (k_dim == 128) return x8 ? launch<128, 128, true>(p, s) : launch<128, 128, false>(p, s);
    return x8 ? launch<192, 128, true>(p, s) : launch<192, 128, false>(p, s);
}
