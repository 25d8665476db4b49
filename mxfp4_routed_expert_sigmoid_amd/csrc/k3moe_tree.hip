// Attention of drafted tokens over the paged cache (k3moe_tree_attention): per
// sequence, drafted token i and query head
//   out = sum_j e^(s_j) v_j / sum_j e^(s_j),  s_j = scale q_i . k_j,
// over the context and the drafted tokens whose bits are set in i's word.
//
// The rows that share a key/value head, (token, head of the group), are one
// matrix: 32 or 128 of them per block. The work is a line of units, a unit being
// 64 keys of one (sequence, key/value head, block of rows), cut into equal runs,
// one per block, so that sequences of any lengths fill the card alike. What a run
// holds whole is written at once; cut ends (two per block at most) go to the
// workspace as unnormalised sums with their maximum, and a second kernel joins
// them in their order.
//
// Up to 32 rows (k_tree_few; 64, in two blocks, over 8 bits) are bound by the
// cache's bytes: every wave holds all rows of its block and reads tiles of 32
// keys of its own, every fourth of the run, through its own part of the LDS, so
// nothing waits for another wave until a segment ends and the four waves' sums
// are added. 32 sequences of up to 32768 tokens, 8 heads of 128: 395 us in bf16
// (2.3 GB, 5.9 TB/s), 222 over 8 bits (5.4 TB/s; there the expansion, two
// operations per value with its LDS write, is as long as the loads). One
// sequence of 4000: 8.7 us and the join's 4.5, the ends of two short kernels.
// Heads of 64, 32 sequences: 207 us (1.16 GB, 5.6 TB/s). Heads of 192 / 128 over 8
// bits do not fit the 256 registers that two blocks on a CU leave a lane: 42 spill
// (156 bytes a lane), and 16 sequences of up to 8000 tokens take 30 us and the
// join's 5 (bf16, one block per CU and no spill, 48 in all for twice the bytes).
//
// More rows (k_tree_wide) are split over the waves, which share tiles of 64 keys
// as the prompts' kernel does. 64 keys of 128 rows take 1.5 us, the time of one
// wave's products and exponentials, which no second wave on its SIMD fills: three
// tiles take the LDS, the accumulators the registers. Plan, first tiles and the
// stores of cut ends are another 10 us. 6 sequences of 16 drafted tokens over up
// to 5000 keys: 34 us and the join's 4.5.
//
// Two launches, no counters: a workspace need not hold anything in front of a
// call, and no block waits for another.
#include "k3moe_attn.h"

namespace k3moe {
namespace {

constexpr int kTrWaves = 4, kTrTile = 32;   // keys of a wave's tile
constexpr int kTrLeast = 2;                 // units of a run at least: a tile for each wave
constexpr int kTrMaxDraft = 64;             // bits of a word
constexpr int kTrMaxRuns = 512, kTrMaxRows = 128, kTrFew = 32;
constexpr int kTrCus = 256, kTrMaxRunRows = kTrCus * kTrMaxRows;   // 512 runs have 32 rows each, 256 have up to 128
static_assert(kTrMaxRuns * kTrFew <= kTrMaxRunRows, "rows of all runs");

// A segment whose runs k_tree_join joins, left by the first run that begins within it (last < 0: no such run).
struct TreeCut {
    int first, last;            // its runs
    int q0, n, kvh, rows0;      // its sequence's rows, its head, its first row (token, head of the group)
};

struct TreeParams {
    const uint16_t *q;
    const uint8_t *kc, *vc, *ks, *vs;
    const int32_t *pages, *lens, *cu;
    const uint64_t *tree;
    uint16_t *out;
    float *lse, *part, *ml;   // part [2 runs][rows][DV], ml [2 runs][rows][2]
    TreeCut *cut;             // [runs]
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

// The line of units and a block's run of it. Runs of `per` units follow each other regardless of segments (a segment:
// the units of one sequence, head and block of rows), or, where the runs of segments cut on their own fit the blocks
// too, begin with the segments: a block then has one segment instead of up to two ends, one after the other.
struct TreePlan {
    int total, per, own;        // own: runs begin with segments
    int b, seg, tile, last;     // where the run begins: sequence, segment in it, tile; units of the run (0: none)
    TreeSeq s;
};

__device__ __forceinline__ TreeSeq tree_pick(const TreeSeq &s, int l)
{
    TreeSeq r;
    r.q0 = __builtin_amdgcn_readlane(s.q0, l), r.n = __builtin_amdgcn_readlane(s.n, l);
    r.ctx = __builtin_amdgcn_readlane(s.ctx, l), r.keys = __builtin_amdgcn_readlane(s.keys, l);
    r.kt = __builtin_amdgcn_readlane(s.kt, l), r.rt = __builtin_amdgcn_readlane(s.rt, l);
    r.units = __builtin_amdgcn_readlane(s.units, l);
    return r;
}

__device__ __forceinline__ TreePlan tree_plan(const TreeParams &p, int number)
{
    const int lane = threadIdx.x & 63;
    TreePlan r{};
    TreeSeq s{};
    int upto = 0;
    for (int b0 = 0; b0 < p.seqs; b0 += 64) {
        s = tree_seq(p, b0 + lane);
        upto = wave_scan(s.units) + r.total;
        r.total = __builtin_amdgcn_readlane(upto, 63);
    }
    r.per = max((r.total + p.runs - 1) / p.runs, kTrLeast);
    if (p.seqs <= 64) {
        // the smallest length, of the first few, with which every segment's own runs fit
        const int segs = s.units > 0 ? p.Hkv * s.rt : 0;
        for (int more = 0; more < 4 && !r.own; ++more) {
            const int per = r.per + more, runs = segs > 0 ? (s.kt + per - 1) / per : 0;
            const int sum = wave_scan(segs * runs), all = __builtin_amdgcn_readlane(sum, 63);
            // (at most one run per unit, so that the sum fits 32 bits too)
            if (all > p.runs) continue;
            r.own = 1, r.per = per;
            if (number >= all) return r;
            const int at = __builtin_ctzll(__ballot(sum > number));
            const int in = number - __builtin_amdgcn_readlane(sum - segs * runs, at), each = __builtin_amdgcn_readlane(runs, at);
            r.b = at, r.s = tree_pick(s, at), r.seg = in / each, r.tile = (in - r.seg * each) * per;
            r.last = min(per, r.s.kt - r.tile);
            return r;
        }
    }
    const int64_t unit = (int64_t)r.per * number;
    if (unit >= r.total) return r;
    r.last = min(r.per, r.total - (int)unit);
    int before = 0;
    for (int b0 = 0; b0 < p.seqs; b0 += 64) {
        if (p.seqs > 64) {
            s = tree_seq(p, b0 + lane);
            upto = wave_scan(s.units) + before;
        }
        const uint64_t past = __ballot(upto > unit);
        if (past) {
            const int at = __builtin_ctzll(past), in = (int)unit - __builtin_amdgcn_readlane(upto - s.units, at);
            r.b = b0 + at, r.s = tree_pick(s, at), r.seg = in / r.s.kt, r.tile = in - r.seg * r.s.kt;
            return r;
        }
        before = __builtin_amdgcn_readlane(upto, 63);
    }
    return r;
}

// Run `number` begins within a segment, as the first of the segment's: what the join has to know.
__device__ __forceinline__ void tree_cut(const TreeParams &p, const TreePlan &r, int number)
{
    if (threadIdx.x) return;
    TreeCut c{};
    if (r.last > 0 && r.tile > 0 && r.tile <= r.per) {
        c.first = number - 1, c.last = number + (r.s.kt - r.tile - 1) / r.per;
        c.q0 = r.s.q0, c.n = r.s.n, c.kvh = r.seg / r.s.rt, c.rows0 = (r.seg - c.kvh * r.s.rt) * p.rows;
    } else {
        c.last = -1;
    }
    p.cut[number] = c;
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
    // Whether a group's byte is 255 in any lane; such a group is zero, whatever its codes.
    __device__ __forceinline__ uint32_t top() const
    {
        uint32_t m = sc[0];
#pragma unroll
        for (int i = 1; i < L; ++i) m = max(m, sc[i]);
        return m;
    }
    __device__ __forceinline__ void drop()
    {
#pragma unroll
        for (int i = 0; i < L; ++i) w[i] = sc[i] == 255u ? u4{0u, 0u, 0u, 0u} : w[i];
    }
    // As bf16 into rows row0 .. row0 + 15 of a tile.
    template <class Slot>
    __device__ __forceinline__ void store(uint8_t *tile, int row0, Slot slot) const
    {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int at = 64 * i + lane, row = row0 + at / (D / 16), sub = at % (D / 16);
            const float f = e8m0_to_f32(sc[i]);
            const u4 x = w[i];
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

// A lane's row of a block: (token, head of the group), with what it sees.
struct TreeRow {
    int64_t token;
    int head;
    bool have;
    uint64_t word;

    __device__ __forceinline__ TreeRow(const TreeParams &p, const TreeSeq &s, int kvh, int m)
    {
        have = m < s.n * p.group;
        const int i = min(m / p.group, s.n - 1);
        token = s.q0 + i, head = kvh * p.group + m % p.group;
        word = (p.tree ? p.tree[token] : low_bits(i + 1)) & low_bits(s.n);
    }
    // which of the 64 keys from `first` on it sees, whatever their pages
    __device__ __forceinline__ uint64_t seen(const TreeSeq &s, int first) const
    {
        const int a = s.ctx - first;   // those in front of the drafted ones
        const uint64_t drafted = a >= 64 || a <= -64 ? 0ull : a >= 0 ? word << a : word >> -a;
        return (low_bits(a) | drafted) & low_bits(s.keys - first);
    }
    // Stores N values of the row from register e0 of its lane on (register e: dimension 32 (e / 16) + 8 (e % 16 / 4) +
    // 4 h + e % 4), or leaves them in the workspace where tiles t0 .. t1 are not all of the segment's. M: the maximum,
    // in powers of two; L: the sum; at: the row's place in the block.
    template <int DV, int N>
    __device__ __forceinline__ void store(const TreeParams &p, const TreeSeq &s, const float (&v)[N], int e0, float M, float L,
                                          int t0, int t1, int at) const
    {
        const int h = (threadIdx.x & 63) >> 5;
        if (!have) return;
        if (t0 == 0 && t1 == s.kt) {
            const float inv = L == 0.0f ? 0.0f : 1.0f / L;
            if (p.lse && h == 0 && e0 == 0) p.lse[token * p.Hq + head] = L == 0.0f ? -INFINITY : (M + __log2f(L)) * kLn2;
            uint16_t *op = p.out + token * p.os + (int64_t)head * DV + 4 * h;
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const int e = e0 + i;
                *reinterpret_cast<uint2 *>(op + 32 * (e >> 4) + 2 * (e & 15)) =
                    uint2{at_bf16(v[i] * inv) | (at_bf16(v[i + 1] * inv) << 16), at_bf16(v[i + 2] * inv) | (at_bf16(v[i + 3] * inv) << 16)};
            }
        } else {
            // a segment cut in front goes to the block's first place, one cut behind only to its second
            const int64_t to = (int64_t)(2 * (int)blockIdx.x + (t0 == 0)) * p.rows + at;
            float *op = p.part + to * DV + 4 * h;
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const int e = e0 + i;
                *reinterpret_cast<float4 *>(op + 32 * (e >> 4) + 2 * (e & 15)) = float4{v[i], v[i + 1], v[i + 2], v[i + 3]};
            }
            if (h == 0 && e0 == 0) *reinterpret_cast<float2 *>(p.ml + 2 * to) = float2{M, L};
        }
    }
};

template <int DK, int DV, bool X8>
struct TreeShape {
    static constexpr int KB = kTrTile * DK * 2, VB = kTrTile * DV * 2;   // a wave's tile
    static constexpr int kBufs = X8 ? 1 : 2;
    static constexpr int kTiles = kTrWaves * kBufs * (KB + VB), kSums = kTrWaves * (DV / 2 + 1) * 64 * 4;
    static constexpr int kLds = kTiles > kSums ? kTiles : kSums;          // the waves' sums take the tiles' place
    static constexpr int kPerCu = kLds <= 80 * 1024 ? 2 : 1;             // blocks that fit a CU
    static_assert(kTrCus * kPerCu <= kTrMaxRuns, "runs");
};

template <int DK, int DV, bool X8>
__global__ __launch_bounds__(64 * kTrWaves, (TreeShape<DK, DV, X8>::kPerCu)) void k_tree_few(TreeParams p)
{
#ifdef __HIP_DEVICE_COMPILE__
    typedef TreeShape<DK, DV, X8> S;
    constexpr int KB = S::KB, VB = S::VB, EB = X8 ? 1 : 2;
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5, l32 = lane & 31;
    const TreePlan plan = tree_plan(p, (int)blockIdx.x);
    tree_cut(p, plan, (int)blockIdx.x);
    if (plan.last <= 0) return;
    int left = plan.last, b = plan.b, seg = plan.seg, t0 = plan.tile;
    TreeSeq s = plan.s;
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
        // tiles t0 .. t1 (of 64 keys) of segment seg of sequence b
        const int kvh = seg / s.rt, rows0 = (seg - kvh * s.rt) * kTrFew;
        const int t1 = min(s.kt, t0 + left);
        const int j1 = min(2 * t1, (s.keys + kTrTile - 1) / kTrTile);   // tiles of 32 keys

        const TreeRow row(p, s, kvh, rows0 + l32);
        v16f o[DV / 32];
        float mx = -INFINITY, l = 0.0f;
#pragma unroll
        for (int d = 0; d < DV / 32; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;

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
        const uint8_t *kt = mine, *vt = mine + KB;
        bool whole = false;                                // every row sees the whole tile
        // Makes tile j ready at kt, vt and sends for the next one.
        auto ready = [&]() {
            ok = ok_next;
            const bool more = j + kTrWaves < j1;
            if constexpr (X8) {
                wave_lds_sync();                           // the last tile is read
                if (__ballot(max(max(bk[0].top(), bk[1].top()), max(bv[0].top(), bv[1].top())) == 255u)) {
#pragma unroll
                    for (int g = 0; g < 2; ++g) bk[g].drop(), bv[g].drop();
                }
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    bk[g].store(mine, 16 * g, k_slot<DK>);
                    bv[g].store(mine + KB, 16 * g, v_slot<DV>);
                }
                if (more) load(j + kTrWaves, 0);
                wave_lds_sync();
            } else {
                kt = mine + buf * (KB + VB), vt = kt + KB;
                buf ^= 1;
                if (more) {
                    wave_lds_sync();                       // the other buffer is read
                    load(j + kTrWaves, buf);
                    wait_loads<2 * (DK + DV) / 32>();
                } else {
                    wait_loads<0>();
                }
            }
            whole = (j + 1) * kTrTile <= s.ctx && ok == ~0u;
        };
        v16f sc;
        bf8 q[DK / 16], pw[2];
        auto scores = [&]() {
            const uint32_t at = fresh(krow), x = fresh(kx);
#pragma unroll
            for (int i = 0; i < 16; ++i) sc[i] = 0.0f;
#pragma unroll
            for (int k = 0; k < DK / 16; ++k)
                sc = mfma32(as_bf8(*reinterpret_cast<const u4 *>(kt + at + (x ^ (32u * k)))), q[k], sc);
        };
        auto weights = [&]() {
            float m = sc[0];
#pragma unroll
            for (int i = 1; i < 16; ++i) m = fmaxf(m, sc[i]);
            m = in_powers(swap_max(m), c);
            const bool up = raises(m, mx);                 // as att_raise: the other rows keep theirs
            if (__ballot(up)) {
                const float f = up ? raised_by(mx, m) : 1.0f;
                mx = up ? m : mx, l *= f;
#pragma unroll
                for (int d = 0; d < DV / 32; ++d)
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[d][i] *= f;
            }
            const float mc = mx == -INFINITY ? 0.0f : mx;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                sc[i] = __builtin_amdgcn_exp2f(fmaf(sc[i], c, -mc));
                l += sc[i];
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)
                pw[k] = as_bf8(u4{at_pack(sc[8 * k], sc[8 * k + 1]), at_pack(sc[8 * k + 2], sc[8 * k + 3]),
                                  at_pack(sc[8 * k + 4], sc[8 * k + 5]), at_pack(sc[8 * k + 6], sc[8 * k + 7])});
        };
        auto values = [&]() {
            const uint32_t from = fresh(vrow), x = fresh(vx);
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int d = 0; d < DV / 32; ++d) {
                    const uint8_t *at = vt + from + (x ^ (64u * d)) + 32 * k * DV;
                    const s4 a0 = lds_tr(at), a1 = lds_tr(at + 16 * DV);
                    bf8 a;
                    __builtin_memcpy(&a, &a0, 8);
                    __builtin_memcpy(reinterpret_cast<char *>(&a) + 8, &a1, 8);
                    o[d] = mfma32(a, pw[k], o[d]);
                }
        };
        if (j < j1) {
            look(j);
            load(j, 0);
            const uint16_t *qp = p.q + row.token * p.qs + (int64_t)row.head * DK + 8 * h;
#pragma unroll
            for (int k = 0; k < DK / 16; ++k) q[k] = as_bf8(*reinterpret_cast<const u4 *>(qp + 16 * k));
        }
        while (j < j1) {
            ready();
            while (whole) {
                scores();
                weights();
                values();
                j += kTrWaves;
                if (j >= j1) break;
                ready();
            }
            if (j >= j1) break;
            scores();
            const uint32_t seen = (uint32_t)row.seen(s, j * kTrTile) & ok;
#pragma unroll
            for (int i = 0; i < 16; ++i) sc[i] = (seen >> (4 * h)) & (1u << (8 * (i >> 2) + (i & 3))) ? sc[i] : -INFINITY;
            weights();
            if (v_not_finite<DV, kTrTile>(vt)) {
                // the rows that see such values get them here; the tile, this wave's own, goes on without them
                att_not_finite<DV>(o, sc, vt, 0, seen);
#pragma unroll 1
                for (int i = 0; i < VB / 1024; ++i) {
                    u4 *at = reinterpret_cast<u4 *>(const_cast<uint8_t *>(vt) + 1024 * i + 16 * lane);
                    const bf8 clean = only_finite(as_bf8(*at));
                    __builtin_memcpy(at, &clean, 16);
                }
                wave_lds_sync();
            }
            values();
            j += kTrWaves;
        }

        // The four waves' sums: all rows' maxima first, then each wave adds a quarter of the dimensions.
        constexpr int R = DV / 2, RW = R / kTrWaves;       // a row's values per lane, and per wave
        float *sums = reinterpret_cast<float *>(lds), *ml = sums + kTrWaves * R * 64;
        const float lw = l + __shfl_xor(l, 32);
        at_barrier();                                      // the tiles are read
        if (h == 0) ml[wave * 64 + l32] = mx, ml[wave * 64 + 32 + l32] = lw;
        at_barrier();
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kTrWaves; ++w) M = fmaxf(M, ml[w * 64 + l32]);
        float L = 0.0f, f = 0.0f;
#pragma unroll
        for (int w = 0; w < kTrWaves; ++w) {
            const float m = ml[w * 64 + l32], x = ml[w * 64 + 32 + l32];
            const float g = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - M);
            L += m == -INFINITY ? x : x * g;               // without a score above -inf: 0, or NaN
            f = w == wave ? g : f;
        }
#pragma unroll
        for (int d = 0; d < DV / 32; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) sums[(wave * R + 16 * d + i) * 64 + lane] = o[d][i] * f;
        at_barrier();
        float v[RW];
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            v[i] = 0.0f;
#pragma unroll
            for (int w = 0; w < kTrWaves; ++w) v[i] += sums[(w * R + RW * wave + i) * 64 + lane];
        }
        row.store<DV, RW>(p, s, v, RW * wave, M, L, t0, t1, l32);

        left -= t1 - t0;
        if (left <= 0) return;
        at_barrier();                                      // the sums are read
        t0 = 0;
        if (++seg == p.Hkv * s.rt) {
            seg = 0;
            do s = tree_seq(p, ++b);
            while (s.units == 0 && b < p.seqs);
            if (b >= p.seqs) return;                       // the lengths have changed meanwhile
        }
    }
#endif
}

// More rows than 32: 128 per block, 32 per wave, over shared tiles of 64 keys; a wave fetches 16 keys of each, two steps
// before their use: bf16 by direct loads into three buffers, 8 bits through registers, a step in each.
template <int DK, int DV, bool X8>
struct WideShape {
    static constexpr int kBufs = X8 ? 2 : 3;
    static constexpr int kLds = kBufs * kAtKeys * (DK + DV) * 2;
};

template <int DK, int DV, bool X8>
__global__ __launch_bounds__(64 * kTrWaves, 1) void k_tree_wide(TreeParams p)
{
#ifdef __HIP_DEVICE_COMPILE__
    constexpr int KB = kAtKeys * DK * 2, VB = kAtKeys * DV * 2;
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5, l32 = lane & 31;
    const TreePlan plan = tree_plan(p, (int)blockIdx.x);
    tree_cut(p, plan, (int)blockIdx.x);
    if (plan.last <= 0) return;
    int left = plan.last, b = plan.b, seg = plan.seg, t0 = plan.tile;
    TreeSeq s = plan.s;
    const int page = 1 << p.lpage;
    const float c = p.scale * kLog2e;
    RowStage<DK, true> sk;
    RowStage<DV, false> sv;
    ByteStage<DK> bk;
    ByteStage<DV> bv;
    if constexpr (!X8) sk.init(DK), sv.init(DV);

    while (true) {
        const int kvh = seg / s.rt, rows0 = (seg - kvh * s.rt) * kTrMaxRows;
        const int n = min(s.kt - t0, left);                        // tiles of this segment here
        const TreeRow row(p, s, kvh, rows0 + kAtRows * wave + l32);
        const bool busy = rows0 + kAtRows * wave < s.n * p.group;
        // Page numbers of 16 tiles, four (of 16 keys) each, a lane holds one; -1: no such key or page. i counts tiles from t0.
        const int32_t *table = p.pages + (int64_t)b * p.width;
        int ids = -1, ids_from = 0;
        auto look = [&](int i) {
            ids_from = i;
            const int64_t pos = (int64_t)(t0 + i) * kAtKeys + 16 * lane;
            ids = pos < s.keys ? table[pos >> p.lpage] : -1;
            if (ids >= p.n_pages) ids = -1;
        };
        // where this wave's 16 rows of tile i lie, and how many there are
        auto rows_of = [&](int i, int64_t &at) {
            const int id = __builtin_amdgcn_readlane(ids, 4 * (i - ids_from) + wave), pos = (t0 + i) * kAtKeys + 16 * wave;
            at = ((int64_t)max(id, 0) * p.Hkv + kvh) * page + (pos & (page - 1));
            return id < 0 ? 0 : min(s.keys - pos, 16);
        };
        // which of a tile's four runs of 16 keys are in the cache, and the same for its keys
        auto cached = [&](int i) { return (uint32_t)(__ballot(ids >= 0) >> (4 * (i - ids_from))) & 15u; };
        auto keys_of = [](uint32_t runs) {
            uint64_t m = 0;
#pragma unroll
            for (int g = 0; g < 4; ++g) m |= runs >> g & 1 ? 0xffffull << (16 * g) : 0ull;
            return m;
        };
        constexpr int NB = WideShape<DK, DV, X8>::kBufs;
        auto ktile = [&](int i) { return lds + (unsigned)(i + NB) % NB * KB; };
        auto vtile = [&](int i) { return lds + NB * KB + (unsigned)(i + NB) % NB * VB; };
        int64_t kat = 0;
        int krows = 0;                                             // of the keys that were fetched last
        uint32_t ok = 0, ok1 = 0, ok2 = 0, ok3 = 0;                // cached runs of the next three tiles, and of what is fetched
        // Step i's fetches, behind its barrier: keys of tile i + 3, values of tile i + 2. Keys run a tile ahead of the
        // values: step i computes the scores of tile i + 1.
        auto fetch = [&](int i) {
            if constexpr (X8) {                                    // what the last step fetched
                if (__ballot(max(bk.top(), bv.top()) == 255u)) bk.drop(), bv.drop();
                if (i + 2 >= 0 && i + 2 < n) bk.store(ktile(i + 2), 16 * wave, k_slot<DK>);
                if (i + 1 >= 0 && i + 1 < n) bv.store(vtile(i + 1), 16 * wave, v_slot<DV>);
            }
            if (i + 2 >= 0 && i + 2 < n) {
                if constexpr (X8) bv.load(p.vc + kat * DV, p.vs + kat * (DV / 32), krows);
                else sv.load(reinterpret_cast<const uint16_t *>(p.vc) + kat * DV, DV, krows, vtile(i + 2) + 16 * wave * DV * 2);
            }
            if (i + 3 < n) {
                if (i + 3 >= ids_from + 16) look(i + 3);
                ok3 = cached(i + 3);
                krows = rows_of(i + 3, kat);
                if constexpr (X8) bk.load(p.kc + kat * DK, p.ks + kat * (DK / 32), krows);
                else sk.load(reinterpret_cast<const uint16_t *>(p.kc) + kat * DK, DK, krows, ktile(i + 3) + 16 * wave * DK * 2);
            }
            ok = ok1, ok1 = ok2, ok2 = ok3;                        // now of tiles i + 1 .. i + 3
        };
        // In front of step i: keys of tile i + 1 and values of tile i are there; what step i - 1 fetched may be on its way.
        auto step_barrier = [&](int i) {
            if (!X8 && i + 2 < n) {
                asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((DK + DV) / 32) : "memory");
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
            } else if (X8) {
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
            } else {
                at_barrier();
            }
        };
        look(0);
        at_barrier();                                              // the last segment's tiles are read
        AttRows<DK, DV> r;
        auto queries = [&]() {
            const uint16_t *qp = p.q + row.token * p.qs + (int64_t)row.head * DK + 8 * h;
#pragma unroll
            for (int k = 0; k < DK / 16; ++k) r.q[k] = as_bf8(*reinterpret_cast<const u4 *>(qp + 16 * k));
        };
        if constexpr (X8) {                                        // as fetch does it, a wait less
            auto keys = [&](int i) {
                krows = rows_of(i, kat);
                bk.load(p.kc + kat * DK, p.ks + kat * (DK / 32), krows);
            };
            auto values = [&]() { bv.load(p.vc + kat * DV, p.vs + kat * (DV / 32), krows); };
            auto drop = [&]() {
                if (__ballot(max(bk.top(), bv.top()) == 255u)) bk.drop(), bv.drop();
            };
            ok = cached(0), ok1 = n > 1 ? cached(1) : 0u, ok2 = n > 2 ? cached(2) : 0u;
            keys(0), values();
            queries();
            drop();
            bk.store(ktile(0), 16 * wave, k_slot<DK>);
            bv.store(vtile(0), 16 * wave, v_slot<DV>);
            if (n > 1) {
                keys(1), values();
                drop();
                bk.store(ktile(1), 16 * wave, k_slot<DK>);
                if (n > 2) keys(2);
            }
        } else {
            fetch(-3);
            queries();
            fetch(-2), fetch(-1);                                  // now ok: tile 0, ok1: tile 1, ok2: tile 2
        }
        r.clear();
        at_barrier();
        if (!busy) {       // a wave without rows fetches its share of the tiles
            for (int i = 0; i < n; ++i) {
                step_barrier(i);
                fetch(i);
            }
        } else {
            v16f sc[2];
            att_scores(sc, r, ktile(0));
            float mx = att_max(sc);
            int i = 0;
            auto whole = [&](int i, uint32_t in) { return (t0 + i + 1) * kAtKeys <= s.ctx && in == 15u; };
            while (i < n) {
                while (i + 1 < n && whole(i, ok) && whole(i + 1, ok1)) {
                    v16f o[2];
                    step_barrier(i);
                    fetch(i);
                    att_tile(r, sc, mx, o, ktile(i + 1), vtile(i), c);
                    step_barrier(i + 1);
                    fetch(i + 1);
                    att_tile(r, o, mx, sc, ktile(i + 2), vtile(i + 1), c);
                    i += 2;
                }
                if (i >= n) break;
                const uint32_t in = ok;
                step_barrier(i);
                fetch(i);
                att_tile_masked(r, sc, ktile(i + 1), vtile(i), c, row.seen(s, (t0 + i) * kAtKeys) & keys_of(in),
                                i + 1 < n);
                mx = att_max(sc);
                ++i;
            }
            const float l = r.l + __shfl_xor(r.l, 32);
            float v[DV / 2];
#pragma unroll
            for (int d = 0; d < DV / 32; ++d)
#pragma unroll
                for (int e = 0; e < 16; ++e) v[16 * d + e] = r.o[d][e];
            row.store<DV, DV / 2>(p, s, v, 0, r.m, l, t0, t0 + n, kAtRows * wave + l32);
        }

        left -= n;
        if (left <= 0) return;
        t0 = 0;
        if (++seg == p.Hkv * s.rt) {
            seg = 0;
            do s = tree_seq(p, ++b);
            while (s.units == 0 && b < p.seqs);
            if (b >= p.seqs) return;                       // the lengths have changed meanwhile
        }
    }
#endif
}

// Joins the cut ends. Block (w, y): where run w + 1 is the first that begins within its segment, some rows of that
// segment, DV / 4 threads for a row.
template <int DV>
__global__ __launch_bounds__(256) void k_tree_join(TreeParams p)
{
    constexpr int TR = DV / 4, RB = 256 / TR;             // threads of a row, rows of a block
    const TreeCut cut = p.cut[blockIdx.x + 1];
    const int row = (int)blockIdx.y * RB + (int)threadIdx.x / TR, part = (int)threadIdx.x % TR;
    const int m = cut.rows0 + row;
    if (cut.last < 0 || m >= cut.n * p.group) return;
    const int base = ((int)threadIdx.x & 63) / TR * TR;   // the row's first lane
    float mx = -INFINITY, l = 0.0f;
    float4 o = float4{0.0f, 0.0f, 0.0f, 0.0f};
    constexpr int G = 16;                                 // runs whose sums are read at a time
    for (int r0 = cut.first; r0 <= cut.last; r0 += G) {
        auto place = [&](int r) { return (int64_t)(2 * r + (r == cut.first)) * p.rows + row; };
        // a thread looks at one run's maximum and sum
        const int r = r0 + part, n = min(G, cut.last - r0 + 1);
        const float2 x = part < n ? *reinterpret_cast<const float2 *>(p.ml + 2 * place(r)) : float2{-INFINITY, 0.0f};
        float4 v[G];
#pragma unroll
        for (int k = 0; k < G; ++k) v[k] = *reinterpret_cast<const float4 *>(p.part + place(r0 + min(k, n - 1)) * DV + 4 * part);
        float top = x.x;
#pragma unroll
        for (int s = 1; s < TR; s <<= 1) top = fmaxf(top, __shfl_xor(top, s));
        top = fmaxf(top, mx);
        const float use = top == -INFINITY ? 0.0f : top;
        const float old = mx == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mx - use);
        const float f = x.x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(x.x - use);
        mx = top;
        l = l * old + (x.x == -INFINITY ? x.y : x.y * f);     // without a score above -inf: 0, or NaN
        o.x *= old, o.y *= old, o.z *= old, o.w *= old;
#pragma unroll
        for (int k = 0; k < G; ++k) {
            const float g = __shfl(f, base + k);              // 0 where there is no such run: its sums count as zeros
            const float4 w = k < n ? v[k] : float4{0.0f, 0.0f, 0.0f, 0.0f};
            o.x = fmaf(w.x, g, o.x), o.y = fmaf(w.y, g, o.y), o.z = fmaf(w.z, g, o.z), o.w = fmaf(w.w, g, o.w);
        }
    }
#pragma unroll
    for (int s = 1; s < TR; s <<= 1) l += __shfl_xor(l, s);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t t = cut.q0 + m / p.group;
    const int head = cut.kvh * p.group + m % p.group;
    *reinterpret_cast<uint2 *>(p.out + t * p.os + (int64_t)head * DV + 4 * part) =
        uint2{at_bf16(o.x * inv) | (at_bf16(o.y * inv) << 16), at_bf16(o.z * inv) | (at_bf16(o.w * inv) << 16)};
    if (p.lse && part == 0) p.lse[t * p.Hq + head] = l == 0.0f ? -INFINITY : (mx + __log2f(l)) * kLn2;
}

template <int DV>
k3moe_status launch(void (*kernel)(TreeParams), int lds, TreeParams p, int per_cu, int rows, hipStream_t s)
{
    p.runs = kTrCus * per_cu, p.rows = rows;
    p.ml = p.part + (size_t)2 * p.runs * p.rows * DV;
    p.cut = reinterpret_cast<TreeCut *>(p.ml + (size_t)2 * p.runs * p.rows * 2);
    kernel<<<(unsigned)p.runs, 64 * kTrWaves, lds, s>>>(p);
    k_tree_join<DV><<<dim3((unsigned)p.runs - 1, (unsigned)(p.rows / (1024 / DV))), 256, 0, s>>>(p);
    return hipGetLastError() == hipSuccess ? K3MOE_OK : K3MOE_E_HIP;
}

template <int DK, int DV, bool X8>
k3moe_status launch(const TreeParams &p, hipStream_t s)
{
    typedef TreeShape<DK, DV, X8> Few;
    typedef WideShape<DK, DV, X8> Wide;
    static std::atomic<uint64_t> few{0}, wide{0};
    // Up to 32 rows a wave that holds them all wins (8 sequences x 4000 keys x 8 heads, 32 rows: 30 us and 35, over 8 bits
    // 27 and 36); behind that two blocks of 32 rows read a bf16 cache twice (40 rows: 47 and 37), but expand an 8-bit one
    // faster than one block of 128, alone on its CU, does (64 rows: 35 and 39; 32 x 8000: 171 and 220; 96 rows: 49 and 42).
    if (p.maxq * p.group <= (X8 ? 2 * kTrFew : kTrFew)) {
        if (!allow_lds(reinterpret_cast<const void *>(k_tree_few<DK, DV, X8>), Few::kLds, few)) return K3MOE_E_HIP;
        return launch<DV>(k_tree_few<DK, DV, X8>, Few::kLds, p, Few::kPerCu, kTrFew, s);
    }
    if (!allow_lds(reinterpret_cast<const void *>(k_tree_wide<DK, DV, X8>), Wide::kLds, wide)) return K3MOE_E_HIP;
    return launch<DV>(k_tree_wide<DK, DV, X8>, Wide::kLds, p, 1, kTrMaxRows, s);
}

template <int DK, int DV>
k3moe_status launch(const TreeParams &p, bool x8, hipStream_t s)
{
    return x8 ? launch<DK, DV, true>(p, s) : launch<DK, DV, false>(p, s);
}

bool at(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

// For the most runs, and the most rows of all runs, that any variant has.
size_t ws_bytes(int v_dim)
{
    return (size_t)2 * kTrMaxRunRows * (size_t)(v_dim + 2) * 4 + kTrMaxRuns * sizeof(TreeCut);
}

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
        cache->pages < 0 || cache->page <= 0 || !(scale > 0.0f && scale <= 0x1p64f))
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
