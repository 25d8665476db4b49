// Attention of drafted tokens over the paged cache (k3moe_tree_attention): per
// sequence, drafted token i and query head
//   out = sum_j e^(s_j) v_j / sum_j e^(s_j),  s_j = scale q_i . k_j,
// over the context and the drafted tokens whose bits are set in i's word.
//
// The rows that share a key/value head, (token, head of the group), are one
// matrix: 32 or 64 of them per block. The work is a line of units, a unit being
// 64 keys of one (sequence, key/value head, block of rows), cut into equal runs,
// one per block, so that sequences of any lengths fill the card alike. What a run
// holds whole is written at once; cut ends (two per block at most) go to the
// workspace as unnormalised sums with their maximum, and a second kernel joins
// them in their order.
//
// Bound by the cache's bytes: every wave holds all rows of its block and reads
// tiles of 32 keys of its own, every fourth of the run, through its own part of
// the LDS, so nothing waits for another wave until a segment ends and the four
// waves' sums are added.
#include "k3moe_attn.h"

namespace k3moe {
namespace {

constexpr int kTrWaves = 4, kTrTile = 32;   // keys of a wave's tile
constexpr int kTrLeast = 2;                 // units of a run at least: a tile for each wave
constexpr int kTrMaxDraft = 64;             // bits of a word
constexpr int kTrMaxRuns = 512, kTrMaxRows = 64;

struct TreeParams {
    const uint16_t *q;
    const uint8_t *kc, *vc, *ks, *vs;
    const int32_t *pages, *lens, *cu;
    const uint64_t *tree;
    uint16_t *out;
    float *lse, *part, *ml;   // part [2 runs][rows][DV], ml [2 runs][rows][2]
    int64_t qs, os;
    int seqs, Tq, maxq, Hq, Hkv, group, n_pages, lpage, width;
    int runs, rows;           // blocks, rows of a block
    float scale;
};

// What a sequence has to do.
struct TreeSeq {
    int q0, n, ctx, keys, kt, rt;   // first row, drafted tokens, context, keys, tiles of keys and blocks of rows
    int units;
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
    s.rt = (s.n * p.group + p.rows - 1) / p.rows;
    s.units = p.Hkv * s.rt * s.kt;                     // the host has checked that their sum fits
    return s;
}

// The sum over the lanes up to and with this one.
__device__ __forceinline__ int wave_scan(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);   // one lane to the right, within a row
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // row 0 into 1, 2 into 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);   // row 1 into 2 and 3
    return v;
}

__device__ __forceinline__ int run_length(const TreeParams &p, int units)
{
    return max((units + p.runs - 1) / p.runs, kTrLeast);
}

// The line of units: its length, the length of a run, and for unit run * number the sequence that holds it with the
// units in front of that sequence (b < 0: the line is shorter). 64 sequences at a time; up to 64 are looked at once.
struct TreePlan {
    int total, per, b, front;
};
__device__ __forceinline__ TreePlan tree_plan(const TreeParams &p, int number)
{
    const int lane = threadIdx.x & 63;
    TreePlan r{0, 0, -1, 0};
    int units = 0, upto = 0;
    for (int b0 = 0; b0 < p.seqs; b0 += 64) {
        units = tree_seq(p, b0 + lane).units;
        upto = wave_scan(units) + r.total;
        r.total = __builtin_amdgcn_readlane(upto, 63);
    }
    r.per = run_length(p, r.total);
    const int64_t unit = (int64_t)r.per * number;
    if (unit >= r.total) return r;
    int before = 0;
    for (int b0 = 0; b0 < p.seqs; b0 += 64) {
        if (p.seqs > 64) {
            units = tree_seq(p, b0 + lane).units;
            upto = wave_scan(units) + before;
        }
        const uint64_t past = __ballot(upto > unit);
        if (past) {
            const int at = __builtin_ctzll(past);
            r.b = b0 + at;
            r.front = __builtin_amdgcn_readlane(upto - units, at);
            return r;
        }
        before = __builtin_amdgcn_readlane(upto, 63);
    }
    return r;
}

#ifdef __HIP_DEVICE_COMPILE__
__device__ __forceinline__ u4 expand_pair(uint32_t lo, uint32_t hi, float f)
{
    const bf2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, f, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, f, true);
    const bf2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, f, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, f, true);
    const bf8 v = bf8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    u4 r;
    __builtin_memcpy(&r, &v, 16);
    return r;
}

// 16 rows of MXFP8 values on their way through registers: 16 codes and their group's byte per lane and load.
template <int D>
struct ByteStage {
    static constexpr int L = D / 64;
    u4 w[L];
    uint32_t sc[L];

    __device__ __forceinline__ void load(const uint8_t *rows, const uint8_t *bytes, int have)
    {
        const int lane = threadIdx.x & 63;
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(rows), 0, kAtOut, 0x00020000);
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(bytes), 0, kAtOut, 0x00020000);
        typedef unsigned u4v __attribute__((ext_vector_type(4)));
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int at = 64 * i + lane, row = at / (D / 16), sub = at % (D / 16);
            const u4v x = __builtin_amdgcn_raw_buffer_load_b128(r, (int)(row < have ? (uint32_t)(16 * at) : kAtOut), 0, 0);
            w[i] = u4{x[0], x[1], x[2], x[3]};
            sc[i] = __builtin_amdgcn_raw_buffer_load_b8(rs, (int)(row < have ? (uint32_t)(row * (D / 32) + sub / 2) : kAtOut), 0, 0);
        }
    }
    // As bf16 into rows row0 .. row0 + 15 of a tile.
    template <class Slot>
    __device__ __forceinline__ void store(uint8_t *tile, int row0, Slot slot) const
    {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int at = 64 * i + lane, row = row0 + at / (D / 16), sub = at % (D / 16);
            const bool drop = sc[i] == 255u;   // such a group is zero, whatever its codes
            const float f = e8m0_to_f32(sc[i]);
            const u4 x = drop ? u4{0u, 0u, 0u, 0u} : w[i];
            *reinterpret_cast<u4 *>(tile + 16 * slot(row, 2 * sub)) = expand_pair(x.x, x.y, f);
            *reinterpret_cast<u4 *>(tile + 16 * slot(row, 2 * sub + 1)) = expand_pair(x.z, x.w, f);
        }
    }
};

template <int N>
__device__ __forceinline__ void wait_loads()   // all but the last N loads
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
#endif

// NC * 32 rows per block.
template <int DK, int DV, bool X8, int NC>
struct TreeShape {
    static constexpr int KB = kTrTile * DK * 2, VB = kTrTile * DV * 2;   // a wave's tile
    static constexpr int kBufs = X8 ? 1 : 2;
    static constexpr int kTiles = kTrWaves * kBufs * (KB + VB), kSums = kTrWaves * (DV / 2 + 1) * 64 * 4;
    static constexpr int kLds = kTiles > kSums ? kTiles : kSums;          // the waves' sums take the tiles' place
    // blocks that fit a CU: by LDS, and by registers where the accumulators leave room for a second wave per SIMD
    static constexpr int kPerCu = kLds <= 80 * 1024 && NC == 1 ? 2 : 1;
};

template <int DK, int DV, bool X8, int NC>
__global__ __launch_bounds__(64 * kTrWaves, (TreeShape<DK, DV, X8, NC>::kPerCu)) void k_tree(TreeParams p)
{
#ifdef __HIP_DEVICE_COMPILE__
    typedef TreeShape<DK, DV, X8, NC> S;
    constexpr int KB = S::KB, VB = S::VB, EB = X8 ? 1 : 2;
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5, l32 = lane & 31;
    const TreePlan plan = tree_plan(p, (int)blockIdx.x);
    if (plan.b < 0) return;
    int u = plan.per * (int)blockIdx.x, b = plan.b, front = plan.front;
    const int end = min(u + plan.per, plan.total);
    TreeSeq s = tree_seq(p, b);
    const int page = 1 << p.lpage;
    const float c = p.scale * kLog2e;
    uint8_t *mine = lds + wave * S::kBufs * (KB + VB);      // this wave's tiles

    // lane parts of the fragments' addresses
    const uint32_t krow = (uint32_t)(l32 * DK * 2), kx = 16u * (uint32_t)(k_slot<DK>(l32, h) - l32 * (DK / 8));
    const int vr = 4 * h + ((lane & 15) >> 2), vcol = (lane & 16) + 4 * (lane & 3);
    const uint32_t vrow = (uint32_t)(vr * DV * 2 + 2 * vcol), vx = 16u * (uint32_t)(v_slot<DV>(vr, 0) - vr * (DV / 8));
    RowStage<DK, true> sk;
    RowStage<DV, false> sv;
    ByteStage<DK> bk[2];
    ByteStage<DV> bv[2];
    if constexpr (!X8) sk.init(DK), sv.init(DV);

    while (true) {
        // the segment that holds unit u: tiles t0 .. t1 (of 64 keys) of (b, kvh, rows)
        const int in = u - front, seg = in / s.kt, t0 = in - seg * s.kt;
        const int kvh = seg / s.rt, rows0 = (seg - kvh * s.rt) * 32 * NC;
        const int t1 = min(s.kt, t0 + (end - u));
        const int j1 = min(2 * t1, (s.keys + kTrTile - 1) / kTrTile);   // tiles of 32 keys

        // this lane's rows: (token, head of the group)
        int tok[NC], head[NC];
        bool have[NC];
        uint64_t word[NC];
        bf8 q[NC][DK / 16];
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            const int m = rows0 + 32 * n + l32;
            have[n] = m < s.n * p.group;
            tok[n] = min(m / p.group, s.n - 1), head[n] = kvh * p.group + m % p.group;
            const uint16_t *qp = p.q + (int64_t)(s.q0 + tok[n]) * p.qs + (int64_t)head[n] * DK + 8 * h;
#pragma unroll
            for (int k = 0; k < DK / 16; ++k) q[n][k] = as_bf8(*reinterpret_cast<const u4 *>(qp + 16 * k));
            word[n] = (p.tree ? p.tree[s.q0 + tok[n]] : low_bits(tok[n] + 1)) & low_bits(s.n);
        }
        v16f o[NC][DV / 32];
        float mx[NC], l[NC];
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            mx[n] = -INFINITY, l[n] = 0.0f;
#pragma unroll
            for (int d = 0; d < DV / 32; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[n][d][i] = 0.0f;
        }

        // Page numbers of this wave's next 32 tiles, two (of 16 keys) each, a lane holds one; -1: no such key or page.
        const int32_t *table = p.pages + (int64_t)b * p.width;
        int ids = -1, ids_from = 0;
        auto look = [&](int j) {
            ids_from = j;
            const int64_t pos = ((int64_t)j + kTrWaves * (lane >> 1)) * kTrTile + 16 * (lane & 1);
            ids = pos < s.keys ? table[pos >> p.lpage] : -1;
            if (ids >= p.n_pages) ids = -1;
        };
        auto id_of = [&](int j, int g) { return __builtin_amdgcn_readlane(ids, 2 * ((j - ids_from) / kTrWaves) + g); };
        uint32_t ok = 0, ok_next = 0;                      // which of a tile's two runs of 16 keys are in the cache
        auto load = [&](int j, int buf) {
            if (j >= ids_from + 32 * kTrWaves) look(j);
            ok_next = 0;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int id = id_of(j, g), pos = j * kTrTile + 16 * g;
                const int rows = id < 0 ? 0 : min(s.keys - pos, 16);
                ok_next |= id < 0 ? 0u : 0xffffu << (16 * g);
                const int64_t row = ((int64_t)max(id, 0) * p.Hkv + kvh) * page + (pos & (page - 1));
                if constexpr (X8) {
                    bk[g].load(p.kc + row * DK, p.ks + row * (DK / 32), rows);
                    bv[g].load(p.vc + row * DV, p.vs + row * (DV / 32), rows);
                } else {
                    uint8_t *at = mine + buf * (KB + VB);
                    sk.load(reinterpret_cast<const uint16_t *>(p.kc + row * DK * EB), DK, rows, at + 16 * g * DK * 2);
                    sv.load(reinterpret_cast<const uint16_t *>(p.vc + row * DV * EB), DV, rows, at + KB + 16 * g * DV * 2);
                }
            }
        };

        int j = 2 * t0 + wave, buf = 0;
        if (j < j1) {
            look(j);
            load(j, 0);
        }
        for (; j < j1; j += kTrWaves) {
            const uint8_t *kt = mine + buf * (KB + VB), *vt = kt + KB;
            ok = ok_next;
            const bool more = j + kTrWaves < j1;
            if constexpr (X8) {
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    bk[g].store(mine, 16 * g, k_slot<DK>);
                    bv[g].store(mine + KB, 16 * g, v_slot<DV>);
                }
                if (more) load(j + kTrWaves, 0);
                wave_lds_sync();
            } else {
                if (more) {
                    wave_lds_sync();                        // the other buffer is read
                    load(j + kTrWaves, buf ^ 1);
                    wait_loads<2 * (DK + DV) / 32>();
                } else {
                    wait_loads<0>();
                }
                buf ^= 1;
            }
            // scores
            v16f sc[NC];
#pragma unroll
            for (int n = 0; n < NC; ++n)
#pragma unroll
                for (int i = 0; i < 16; ++i) sc[n][i] = 0.0f;
#pragma unroll
            for (int k = 0; k < DK / 16; ++k) {
                const bf8 a = as_bf8(*reinterpret_cast<const u4 *>(kt + krow + (kx ^ (32u * k))));
#pragma unroll
                for (int n = 0; n < NC; ++n) sc[n] = mfma32(a, q[n][k], sc[n]);
            }
            const int first = j * kTrTile, ahead = s.ctx - first;   // the tile's keys in front of the drafted ones
            const bool whole = ahead >= kTrTile && ok == ~0u;
            uint32_t seen[NC];
            bool bad = false;
            bf8 pw[NC][2];
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                seen[n] = ~0u;
                if (!whole) {
                    uint64_t see = low_bits(ahead) | (ahead >= 64 || ahead <= -64 ? 0ull : ahead >= 0 ? word[n] << ahead : word[n] >> -ahead);
                    see &= low_bits(s.keys - first);
                    seen[n] = (uint32_t)see & ok;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        sc[n][i] = (seen[n] >> (4 * h)) & (1u << (8 * (i >> 2) + (i & 3))) ? sc[n][i] : -INFINITY;
                }
                float m = sc[n][0];
#pragma unroll
                for (int i = 1; i < 16; ++i) m = fmaxf(m, sc[n][i]);
                m = swap_max(m);
                if (__ballot((m - mx[n]) * c > kAtSlack)) {
                    const float mn = fmaxf(mx[n], m);
                    const float f = mx[n] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((mx[n] - mn) * c);
                    mx[n] = mn, l[n] *= f;
#pragma unroll
                    for (int d = 0; d < DV / 32; ++d)
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[n][d][i] *= f;
                }
                const float mc = mx[n] == -INFINITY ? 0.0f : mx[n] * c;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    sc[n][i] = __builtin_amdgcn_exp2f(fmaf(sc[n][i], c, -mc));
                    l[n] += sc[n][i];
                }
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    pw[n][k] = as_bf8(u4{at_pack(sc[n][8 * k], sc[n][8 * k + 1]), at_pack(sc[n][8 * k + 2], sc[n][8 * k + 3]),
                                         at_pack(sc[n][8 * k + 4], sc[n][8 * k + 5]), at_pack(sc[n][8 * k + 6], sc[n][8 * k + 7])});
            }
            if (!whole) bad = v_not_finite<DV, kTrTile>(vt);
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int d = 0; d < DV / 32; ++d) {
                    const uint8_t *at = vt + (vrow + (vx ^ (64u * d))) + 32 * k * DV;
                    const s4 a0 = lds_tr(at), a1 = lds_tr(at + 16 * DV);
                    bf8 a;
                    __builtin_memcpy(&a, &a0, 8);
                    __builtin_memcpy(reinterpret_cast<char *>(&a) + 8, &a1, 8);
                    if (bad) a = only_finite(a);
#pragma unroll
                    for (int n = 0; n < NC; ++n) o[n][d] = mfma32(a, pw[n][k], o[n][d]);
                }
            if (bad) {
#pragma unroll
                for (int n = 0; n < NC; ++n) att_not_finite<DV>(o[n], sc[n], vt, 0, seen[n]);
            }
            if constexpr (X8) wave_lds_sync();   // the tile is read
        }

        // The four waves' sums: all rows' maxima first, then each wave adds a quarter of the dimensions.
        const bool complete = t0 == 0 && t1 == s.kt;
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            constexpr int R = DV / 2, RW = R / kTrWaves;   // a row's values per lane, and per wave
            float *sums = reinterpret_cast<float *>(lds), *ml = sums + kTrWaves * R * 64;
            const float lw = l[n] + __shfl_xor(l[n], 32);
            at_barrier();                                  // the tiles, or the last sums, are read
            if (h == 0) ml[wave * 64 + l32] = mx[n], ml[wave * 64 + 32 + l32] = lw;
            at_barrier();
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kTrWaves; ++w) M = fmaxf(M, ml[w * 64 + l32]);
            float L = 0.0f, f = 0.0f;
#pragma unroll
            for (int w = 0; w < kTrWaves; ++w) {
                const float m = ml[w * 64 + l32], x = ml[w * 64 + 32 + l32];
                const float g = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((m - M) * c);
                L += m == -INFINITY ? x : x * g;           // without a score above -inf: 0, or NaN
                f = w == wave ? g : f;
            }
#pragma unroll
            for (int d = 0; d < DV / 32; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) sums[(wave * R + 16 * d + i) * 64 + lane] = o[n][d][i] * f;
            at_barrier();
            float v[RW];
#pragma unroll
            for (int i = 0; i < RW; ++i) {
                v[i] = 0.0f;
#pragma unroll
                for (int w = 0; w < kTrWaves; ++w) v[i] += sums[(w * R + RW * wave + i) * 64 + lane];
            }
            // register e of a row holds dimension 32 (e / 16) + 8 (e % 16 / 4) + 4 h + e % 4
            const int e0 = RW * wave;
            if (have[n]) {
                if (complete) {
                    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
                    if (p.lse && h == 0 && wave == 0)
                        p.lse[(int64_t)(s.q0 + tok[n]) * p.Hq + head[n]] = L == 0.0f ? -INFINITY : fmaf(M, c, __log2f(L)) * kLn2;
                    uint16_t *op = p.out + (int64_t)(s.q0 + tok[n]) * p.os + (int64_t)head[n] * DV + 4 * h;
#pragma unroll
                    for (int i = 0; i < RW; i += 4) {
                        const int e = e0 + i;
                        *reinterpret_cast<uint2 *>(op + 32 * (e >> 4) + 2 * (e & 15)) =
                            uint2{at_bf16(v[i] * inv) | (at_bf16(v[i + 1] * inv) << 16), at_bf16(v[i + 2] * inv) | (at_bf16(v[i + 3] * inv) << 16)};
                    }
                } else {
                    // a segment cut in front goes to the block's first place, one cut behind only to its second
                    const int64_t at = (int64_t)(2 * (int)blockIdx.x + (t0 == 0)) * p.rows + 32 * n + l32;
                    float *op = p.part + at * DV + 4 * h;
#pragma unroll
                    for (int i = 0; i < RW; i += 4) {
                        const int e = e0 + i;
                        *reinterpret_cast<float4 *>(op + 32 * (e >> 4) + 2 * (e & 15)) = float4{v[i], v[i + 1], v[i + 2], v[i + 3]};
                    }
                    if (h == 0 && wave == 0) *reinterpret_cast<float2 *>(p.ml + 2 * at) = float2{M * c, L};   // c > 0: -inf stays
                }
            }
        }

        u += t1 - t0;
        if (u >= end) return;
        at_barrier();                                      // the sums are read
        while (u >= front + s.units) {
            front += s.units;
            s = tree_seq(p, ++b);
        }
    }
#endif
}

// Joins the cut ends. Block (w, y): if the end of run w - 1 is the first one within its segment, the rows 16 y .. of
// that segment, four dimensions per thread.
template <int DV>
__global__ __launch_bounds__(256) void k_tree_join(TreeParams p)
{
    constexpr int TR = DV / 4, RB = 256 / TR;             // threads of a row, rows at a time
    const int w = (int)blockIdx.x + 1;
    const TreePlan plan = tree_plan(p, w);
    if (plan.b < 0) return;
    const int u = plan.per * w;
    const TreeSeq s = tree_seq(p, plan.b);
    const int seg = (u - plan.front) / s.kt, u0 = plan.front + seg * s.kt;
    if (u == u0 || u - plan.per > u0) return;             // no cut, or not the segment's first
    const int kvh = seg / s.rt, rows0 = (seg - kvh * s.rt) * p.rows;
    const int w0 = w - 1, w1 = (u0 + s.kt - 1) / plan.per;
    const int row = (int)blockIdx.y * RB + (int)threadIdx.x / TR, e = 4 * ((int)threadIdx.x % TR);
    const int m = rows0 + row;
    if (row >= p.rows || m >= s.n * p.group) return;
    auto place = [&](int r) { return (int64_t)(2 * r + (r == w0 && u0 >= r * plan.per)) * p.rows + row; };
    float mx = -INFINITY;
    for (int r = w0; r <= w1; ++r) mx = fmaxf(mx, p.ml[2 * place(r)]);
    const float use = mx == -INFINITY ? 0.0f : mx;
    float l = 0.0f;
    float4 o = float4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int r = w0; r <= w1; ++r) {
        const int64_t at = place(r);
        const float2 x = *reinterpret_cast<const float2 *>(p.ml + 2 * at);
        const float4 v = *reinterpret_cast<const float4 *>(p.part + at * DV + e);
        const float f = x.x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(x.x - use);
        l += x.x == -INFINITY ? x.y : x.y * f;            // without a score above -inf: 0, or NaN
        o.x = fmaf(v.x, f, o.x), o.y = fmaf(v.y, f, o.y), o.z = fmaf(v.z, f, o.z), o.w = fmaf(v.w, f, o.w);
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t t = s.q0 + m / p.group;
    const int head = kvh * p.group + m % p.group;
    *reinterpret_cast<uint2 *>(p.out + t * p.os + (int64_t)head * DV + e) =
        uint2{at_bf16(o.x * inv) | (at_bf16(o.y * inv) << 16), at_bf16(o.z * inv) | (at_bf16(o.w * inv) << 16)};
    if (p.lse && e == 0) p.lse[t * p.Hq + head] = l == 0.0f ? -INFINITY : (use + __log2f(l)) * kLn2;
}

template <int DK, int DV, bool X8, int NC>
k3moe_status launch(TreeParams p, hipStream_t s)
{
    typedef TreeShape<DK, DV, X8, NC> S;
    static const hipError_t allowed =
        hipFuncSetAttribute(reinterpret_cast<const void *>(k_tree<DK, DV, X8, NC>), hipFuncAttributeMaxDynamicSharedMemorySize, S::kLds);
    if (allowed != hipSuccess) return K3MOE_E_HIP;
    p.runs = 256 * S::kPerCu, p.rows = 32 * NC;
    p.ml = p.part + (size_t)2 * p.runs * p.rows * DV;
    k_tree<DK, DV, X8, NC><<<(unsigned)p.runs, 64 * kTrWaves, S::kLds, s>>>(p);
    k_tree_join<DV><<<dim3((unsigned)p.runs - 1, (unsigned)(p.rows / (1024 / DV))), 256, 0, s>>>(p);
    return hipGetLastError() == hipSuccess ? K3MOE_OK : K3MOE_E_HIP;
}

template <int DK, int DV>
k3moe_status launch(const TreeParams &p, bool x8, hipStream_t s)
{
    const bool few = p.maxq * (int64_t)p.group <= 32;
    if (x8) return few ? launch<DK, DV, true, 1>(p, s) : launch<DK, DV, true, 2>(p, s);
    return few ? launch<DK, DV, false, 1>(p, s) : launch<DK, DV, false, 2>(p, s);
}

bool at(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

// For the most runs and rows that any variant has.
size_t ws_bytes(int v_dim) { return (size_t)2 * kTrMaxRuns * kTrMaxRows * (size_t)(v_dim + 2) * 4; }

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
    // the line of units is counted in 32 bits; rows of a block: 32 at least
    const int64_t tiles = ((int64_t)pages_width * page + kAtKeys - 1) / kAtKeys + 1;
    const int64_t blocks = (int64_t)seqs * kv_heads * (((int64_t)max_q * (q_heads / kv_heads) + 31) / 32);
    if (blocks > INT32_MAX / 2 || tiles * blocks > INT32_MAX / 2) return K3MOE_E_UNSUPPORTED_SHAPE;
    if (!at(q, 16) || !at(out, 16) || q_stride % 8 || out_stride % 8 || !at(cache->k, 16) || !at(cache->v, 16) || !at(pages, 4) ||
        !at(lens, 4) || !at(cu_q, 4) || !at(tree, 8) || !at(lse, 4))
        return K3MOE_E_ALIGNMENT;
    if (!workspace || !at(workspace, 256) || workspace_bytes < ws_bytes(v_dim)) return K3MOE_E_WORKSPACE;
    TreeParams p{};
    p.q = q, p.kc = static_cast<const uint8_t *>(cache->k), p.vc = static_cast<const uint8_t *>(cache->v);
    p.ks = cache->ks, p.vs = cache->vs, p.pages = pages, p.lens = lens, p.cu = cu_q, p.tree = tree, p.out = out, p.lse = lse;
    p.part = static_cast<float *>(workspace);
    p.qs = q_stride, p.os = out_stride, p.seqs = seqs, p.Tq = Tq, p.maxq = max_q, p.Hq = q_heads, p.Hkv = kv_heads;
    p.group = q_heads / kv_heads, p.n_pages = cache->pages, p.lpage = __builtin_ctz((unsigned)page), p.width = pages_width;
    p.scale = scale;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return k_dim == 64 ? launch<64, 64>(p, x8, s) : k_dim == 128 ? launch<128, 128>(p, x8, s) : launch<192, 128>(p, x8, s);
}
