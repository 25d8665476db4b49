// What the attention kernels share: the inner loop over tiles of 64 keys for a
// wave's 32 rows of queries, and the small pieces around it.
//
// Scores are computed transposed, S^T = K Q^T (32x32x16 MFMAs, keys on the
// rows), so that a lane holds scores of one query only: the running maximum
// and sum of a row stay in its two lanes (l and l ^ 32), and the registers
// that hold P^T are, in the order they have, the B operand of O^T = V^T P^T.
// Its A operand V^T comes from the row-major V tile through the LDS transpose
// reads. The order of the 16 keys of one product is free as long as both
// operands agree; it is the score layout's: slot 8h + j of lane half h is key
// 4h + j for j < 4 and key 8 + 4h + j - 4 behind that.
//
// P is rounded to bf16 for the second product: at most 2^-8 of each weight, as
// much again as the result's own rounding where one key has all of it, less where
// the errors of many keys average out (2.2e-3 of the whole against 64 bits where
// exact weights leave 1.6e-3). The matrix unit takes nothing wider at its rate,
// and two halves of each weight would double the second product. The sums l are
// taken of the fp32 values.
//
// What bounds it: per tile of 64 keys and heads of 128 a wave has 32 products
// (1024 cycles of the matrix unit) and 32 scores a lane, each with one
// exponential, at a quarter of the other operations' rate, and four operations
// more. att_tile interleaves the two by hand, a pair of scores to a step: 8192
// causal tokens of 32 heads take 560 us (0.98 PFLOP/s) where the compiler's
// order took 619, 4096 tokens that see every key 275 (1.0). On runs as long as
// these the card's power sets the pace: its clock goes to 1.5 - 2.0 GHz.
#pragma once

#include <atomic>

#include "k3moe_device.h"
#include "k3moe_internal.h"

namespace k3moe {

// Lets a kernel have `bytes` of LDS on the current device; done: the kernel's own, a bit per device.
inline bool allow_lds(const void *kernel, int bytes, std::atomic<uint64_t> &done)
{
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return false;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
    if (done.load(std::memory_order_relaxed) & bit) return true;
    if (hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes) != hipSuccess) return false;
    done.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

typedef float v16f __attribute__((ext_vector_type(16)));
typedef short s4 __attribute__((ext_vector_type(4)));

constexpr int kAtKeys = 64;                // keys per tile
constexpr int kAtRows = 32;                // rows of queries per wave
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// The running maximum is raised only when a tile exceeds it by more than this (in powers of two): the weights then
// stay below 2^8 of what they would be, which neither fp32 sums nor the bf16 weights, rounded relatively, notice.
constexpr float kAtSlack = 8.0f;
// An offset behind the bytes of 16 rows of 2^24 elements at most: read as zeros.
constexpr uint32_t kAtOut = 0xff000000u;

__device__ __forceinline__ uint32_t at_bf16(float f) { return f != f ? 0x7fc0u : bf16_rne_u32(f); }

// Two fp32 -> packed bf16, to nearest even.
__device__ __forceinline__ uint32_t at_pack(float a, float b)
{
    typedef float f2 __attribute__((ext_vector_type(2)));
    const bf2 p = __builtin_convertvector((f2){a, b}, bf2);
    uint32_t r;
    __builtin_memcpy(&r, &p, 4);
    return r;
}

// Position of 16-byte slot s of row r in a tile of D-wide bf16 rows. K tiles are read one slot of 32 rows at a
// time: 16 neighbouring rows touch every bank once. V tiles are read 64 bytes of four neighbouring rows at a time.
template <int D>
__device__ __forceinline__ int k_slot(int r, int s)
{
    return r * (D / 8) + (D == 128 ? s ^ (r & 15) : s ^ ((r >> 1) & 7));
}
template <int D>
__device__ __forceinline__ int v_slot(int r, int s)
{
    static_assert(D == 64 || D == 128, "value widths");
    return r * (D / 8) + (D == 128 ? s ^ ((r & 3) << 2) : s ^ (((r >> 1) & 1) << 2));
}

__device__ __forceinline__ v16f mfma32(const bf8 &a, const bf8 &b, v16f c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// The maximum of lanes l and l ^ 32.
__device__ __forceinline__ float swap_max(float v)
{
#ifdef __HIP_DEVICE_COMPILE__
    const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
#else
    return v;
#endif
}

// LDS transpose read: the 16 lanes of a quarter wave read 4 rows of 16 values (lane i: 4 values of row i / 4), and
// lane i gets column i of the four rows.
__device__ __forceinline__ s4 lds_tr(const uint8_t *at)
{
    typedef __attribute__((address_space(3))) s4 lds_s4;
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)at);
}

// The lowest n bits (n <= 0: none, n >= 64: all).
__device__ __forceinline__ uint64_t low_bits(int n) { return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1; }

#ifdef __HIP_DEVICE_COMPILE__
// 16 bytes per lane from a buffer into LDS at `lds` (the wave's first byte) on, in the lanes' order. Written as an
// instruction: of the builtin the compiler believes that it may write what the transpose reads read, and waits for every
// load in flight in front of them. at_barrier() waits for these loads.
__device__ __forceinline__ void lds_load16(const void *base, uint32_t offset, uint32_t soffset, const uint8_t *lds)
{
    typedef int v4i __attribute__((ext_vector_type(4)));
    const uint64_t a = (uint64_t)base;
    const v4i rsrc = {__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
                      __builtin_amdgcn_readfirstlane((int)((uint32_t)(a >> 32) & 0xffffu)), (int)kAtOut, 0x00020000};
    const uint32_t at = __builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t *)lds);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(at), "v"(offset), "s"(rsrc),
                 "s"(__builtin_amdgcn_readfirstlane((int)soffset))
                 : "memory");   // m0 is no register that the compiler keeps anything in here
}

// Direct loads of 16 rows of one head into their places of an LDS tile laid out by k_slot (K) or v_slot. The places that
// a load fills are 1 KB in order, so each lane fetches the slot that belongs into its own. With row = 8 a + r the
// exchange of slots is the same for a = 0 and 1 but for one bit of the slot's number (k_slot), or at all (v_slot); so a
// load's offset is a lane constant, exchanged, and a wave constant.
template <int D, bool K>
struct RowStage {
    static constexpr int SL = D / 8, L = D / 32;          // slots per row, loads
    static constexpr int J = D == 192 ? 3 : L / 2;        // loads of 8 rows
    uint32_t x[J], at[J];                                  // 16 * the slot, bytes of the row r

    __device__ __forceinline__ static int row(int j) { return (64 * j + (int)(threadIdx.x & 63)) / SL; }
    // stride: elements between rows, at most 2^24
    __device__ __forceinline__ void init(int64_t stride)
    {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int r = row(j), pos = (64 * j + (int)(threadIdx.x & 63)) % SL;
            x[j] = 16u * (uint32_t)((K ? k_slot<D>(r, pos) : v_slot<D == 192 ? 128 : D>(r, pos)) - r * SL);
            at[j] = (uint32_t)r * (uint32_t)stride * 2u;
        }
    }
    // src: the first of the 16 rows; those from `have` on read as zeros. lds: their first place.
    __device__ __forceinline__ void load(const uint16_t *src, int64_t stride, int have, const uint8_t *lds) const
    {
        const bool whole = have >= 16;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int a = i / J, j = i % J;
            uint32_t o = (x[j] ^ (K ? (D == 128 ? 128u : 64u) * a : 0u)) + at[j];
            if (!whole) o = 8 * a + row(j) < have ? o : kAtOut;
            lds_load16(src, o, 8u * a * (uint32_t)stride * 2u, lds + i * 1024);
        }
    }
};
#endif

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

// Waits for this wave's loads and LDS operations, then for the block.
__device__ __forceinline__ void at_barrier()
{
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// A wave's 32 rows: the queries as B operands, running maximum (in powers of two) and sum, O^T.
template <int DK, int DV>
struct AttRows {
    bf8 q[DK / 16];
    v16f o[DV / 32];
    float m, l;      // m: the same in both lanes of a row; l: each lane's own keys
    __device__ __forceinline__ void clear()
    {
        m = -INFINITY, l = 0.0f;
#pragma unroll
        for (int d = 0; d < DV / 32; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
    }
};

// Whether KEYS rows of a V tile in LDS hold a value that is not finite, for the whole wave.
template <int DV, int KEYS>
__device__ __forceinline__ bool v_not_finite(const uint8_t *vt)
{
    typedef unsigned short h2 __attribute__((ext_vector_type(2)));
    const int lane = threadIdx.x & 63;
    h2 most = h2{0, 0};
#pragma unroll
    for (int i = 0; i < KEYS * DV * 2 / 1024; ++i) {
        const u4 w = *reinterpret_cast<const u4 *>(vt + 1024 * i + 16 * lane);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t e = w[j] & 0x7f807f80u;   // the exponents
            h2 x;
            __builtin_memcpy(&x, &e, 4);
            most = __builtin_elementwise_max(most, x);
        }
        if (i % 2) asm volatile("" ::: "memory");   // two loads at a time: the accumulators hold the registers
    }
    return __ballot(most[0] == 0x7f80u || most[1] == 0x7f80u) != 0;
}

// Zeros in the place of values that are not finite.
__device__ __forceinline__ bf8 only_finite(const bf8 &a)
{
    u4 w;
    __builtin_memcpy(&w, &a, 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = (w[i] & 0x7f80u) == 0x7f80u ? w[i] & 0xffff0000u : w[i];
        w[i] = (w[i] & 0x7f800000u) == 0x7f800000u ? w[i] & 0xffffu : w[i];
    }
    return as_bf8(w);
}

// Keeps the compiler from holding what follows from v in registers across the loop over tiles (a tile's addresses
// are a few operations on one register, or fifty registers that the accumulators need).
__device__ __forceinline__ uint32_t fresh(uint32_t v)
{
    asm volatile("" : "+v"(v));
    return v;
}

// The parts of a tile's work. c: scale * log2(e).
//
// Scores of 64 keys: element i of s[t] is key 32 t + 8 (i / 4) + 4 h + i % 4.
template <int DK, int DV>
__device__ __forceinline__ void att_scores(v16f (&s)[2], const AttRows<DK, DV> &r, const uint8_t *kt)
{
    const int lane = threadIdx.x & 63, h = lane >> 5, l32 = lane & 31;
    // k_slot(32 t + l32, 2 k + h) = row part + (slot of k = 0, exchanged with 2 k)
    const uint32_t krow = fresh((uint32_t)(l32 * DK * 2)), kx = fresh(16u * (uint32_t)(k_slot<DK>(l32, h) - l32 * (DK / 8)));
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[t][i] = 0.0f;
#pragma unroll
        for (int k = 0; k < DK / 16; ++k) {
            const u4 a = *reinterpret_cast<const u4 *>(kt + (krow + (kx ^ (32u * k))) + 64 * t * DK);
            s[t] = mfma32(as_bf8(a), r.q[k], s[t]);
        }
    }
}

// -inf for the keys whose bits are not in `seen`.
__device__ __forceinline__ void att_mask(v16f (&s)[2], uint64_t seen)
{
    const uint64_t mine = seen >> (4 * ((threadIdx.x & 63) >> 5));
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            s[t][i] = (uint32_t)(mine >> (32 * t)) & (1u << (8 * (i >> 2) + (i & 3))) ? s[t][i] : -INFINITY;
}

__device__ __forceinline__ float att_max(const v16f (&s)[2])
{
    float mx = s[0][0];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[t][i]);
    return swap_max(mx);
}

// Running maxima are held in powers of two, score * c, so that a score beyond fp32 is an infinity there: -inf is no
// maximum to start from (mx - m is NaN where both are), and +inf makes the row's sums NaN. The product is rounded by
// itself: contracted with the difference behind it, it would not overflow.
__device__ __forceinline__ float in_powers(float score, float c)
{
#pragma clang fp contract(off)
    return score * c;
}
__device__ __forceinline__ bool raises(float mx, float m) { return mx - m > kAtSlack; }
// What raising m to mx turns the sums by: 0 from -inf on.
__device__ __forceinline__ float raised_by(float m, float mx) { return mx == INFINITY ? NAN : __builtin_amdgcn_exp2f(m - mx); }

// Raises the running maximum of the rows where a score exceeds it by the slack; the others keep theirs, so that a row's
// bits do not depend on what other rows see. mx: the largest raw score.
template <int DK, int DV>
__device__ __forceinline__ void att_raise(AttRows<DK, DV> &r, float mx, float c)
{
    mx = in_powers(mx, c);
    const bool up = raises(mx, r.m);
    if (__ballot(up)) {
        const float a = up ? raised_by(r.m, mx) : 1.0f;
        r.m = up ? mx : r.m, r.l *= a;
#pragma unroll
        for (int d = 0; d < DV / 32; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) r.o[d][i] *= a;
    }
}

// Scores to weights, their sum, and the weights as B operands of the four products with 16 values.
template <int DK, int DV>
__device__ __forceinline__ void att_weights(bf8 (&p)[4], AttRows<DK, DV> &r, v16f (&s)[2], float c)
{
    const float mc = r.m == -INFINITY ? 0.0f : r.m;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            s[t][i] = __builtin_amdgcn_exp2f(fmaf(s[t][i], c, -mc));
            r.l += s[t][i];
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
            p[2 * t + j] = as_bf8(u4{at_pack(s[t][8 * j], s[t][8 * j + 1]), at_pack(s[t][8 * j + 2], s[t][8 * j + 3]),
                                     at_pack(s[t][8 * j + 4], s[t][8 * j + 5]), at_pack(s[t][8 * j + 6], s[t][8 * j + 7])});
    }
}

// O^T += V^T P^T; FINITE: without the values that are not finite.
template <bool FINITE, int DK, int DV>
__device__ __forceinline__ void att_values(AttRows<DK, DV> &r, const bf8 (&p)[4], const uint8_t *vt)
{
    const int lane = threadIdx.x & 63, h = lane >> 5;
    const int vr = 4 * h + ((lane & 15) >> 2), vc = (lane & 16) + 4 * (lane & 3);   // row and column of k = d = 0
    const uint32_t vrow = fresh((uint32_t)(vr * DV * 2 + 2 * vc)), vx = fresh(16u * (uint32_t)(v_slot<DV>(vr, 0) - vr * (DV / 8)));
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int d = 0; d < DV / 32; ++d) {
            const uint8_t *at = vt + (vrow + (vx ^ (64u * d))) + 32 * k * DV;
            const s4 a0 = lds_tr(at), a1 = lds_tr(at + 16 * DV);
            bf8 a;
            __builtin_memcpy(&a, &a0, 8);
            __builtin_memcpy(reinterpret_cast<char *>(&a) + 8, &a1, 8);
            if constexpr (FINITE) a = only_finite(a);
            r.o[d] = mfma32(a, p[k], r.o[d]);
        }
}

// A weight of zero does not hide an infinity or a NaN in a product. Where a tile that not every row sees holds one, the
// products are taken without such values (only_finite), and this adds them to the rows that see them, one by one.
// s: the weights of 32 keys from `key0` of the tile on, bit j of `seen`: whether this lane's row sees the j-th of them.
template <int DV>
__device__ __forceinline__ void att_not_finite(v16f (&o)[DV / 32], const v16f &s, const uint8_t *vt, int key0, uint32_t seen)
{
    const int lane = threadIdx.x & 63, h = lane >> 5;
#pragma unroll 1
    for (int j = 0; j < 16; ++j) {
        float own = s[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) own = j == i ? s[i] : own;
        own = bf16f(at_bf16(own));
        asm volatile("" ::: "memory");
        const float other = __shfl_xor(own, 32);
#pragma unroll 1
        for (int hh = 0; hh < 2; ++hh) {
            const int key = 8 * (j >> 2) + 4 * hh + (j & 3);
            const float w = hh == h ? own : other;
            const bool sees = seen >> key & 1;
#pragma unroll
            for (int d = 0; d < DV / 32; ++d)
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const int col = 32 * d + 2 * i + 4 * h;
                    const uint2 v = *reinterpret_cast<const uint2 *>(vt + 16 * v_slot<DV>(key0 + key, col >> 3) + 2 * (col & 7));
                    const float f[4] = {bf16f(v.x & 0xffffu), bf16f(v.x >> 16), bf16f(v.y & 0xffffu), bf16f(v.y >> 16)};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[d][i + e] = sees && !(fabsf(f[e]) < INFINITY) ? fmaf(w, f[e], o[d][i + e]) : o[d][i + e];
                    asm volatile("" ::: "memory");   // a few values at a time: this path sets no register's limit
                }
        }
    }
}

// One tile whose scores s are there with their maximum mx, on a wave's rows, and the scores of the next tile (nk: its
// keys) with theirs. Every row sees the whole tile. The products of the next scores, which do not depend on this tile's
// weights, carry the exponentials in their shadow, and the products with the values the next maximum; fragments are read
// some steps ahead. The steps are kept in this order: left to itself the compiler takes all exponentials first, then the
// products.
template <int DK, int DV>
__device__ __forceinline__ void att_tile(AttRows<DK, DV> &r, v16f (&s)[2], float &mx, v16f (&next)[2], const uint8_t *nk,
                                         const uint8_t *vt, float c)
{
    constexpr int QS = DK / 8, VS = DV / 8;                 // steps: one product each
    constexpr int QP = (16 + QS - 1) / QS, VP = 16 / VS;    // pairs of scores per step
    constexpr int QA = 4, VA = 3;                           // steps that fragments are read ahead
    const int lane = threadIdx.x & 63, h = lane >> 5, l32 = lane & 31;
    const uint32_t krow = fresh((uint32_t)(l32 * DK * 2)), kx = fresh(16u * (uint32_t)(k_slot<DK>(l32, h) - l32 * (DK / 8)));
    const int vr = 4 * h + ((lane & 15) >> 2), vc = (lane & 16) + 4 * (lane & 3);
    const uint32_t vrow = fresh((uint32_t)(vr * DV * 2 + 2 * vc)), vx = fresh(16u * (uint32_t)(v_slot<DV>(vr, 0) - vr * (DV / 8)));
    u4 ka[QS];
    s4 va[VS][2];
    auto kread = [&](int i) {
        ka[i] = *reinterpret_cast<const u4 *>(nk + (krow + (kx ^ (32u * (i % (DK / 16))))) + 64 * (i / (DK / 16)) * DK);
    };
    auto vread = [&](int i) {
        const uint8_t *at = vt + (vrow + (vx ^ (64u * (i % (DV / 32))))) + 32 * (i / (DV / 32)) * DV;
        va[i][0] = lds_tr(at), va[i][1] = lds_tr(at + 16 * DV);
    };
#pragma unroll
    for (int i = 0; i < QA; ++i) kread(i);
    att_raise(r, mx, c);
    const float mc = r.m == -INFINITY ? 0.0f : r.m;
    uint32_t p[16];
    float l[2] = {r.l, 0.0f};
    // a pair of scores goes through its operations a step apart each, so that none waits for the one in front of it
    auto scaled = [&](int w) {
#pragma unroll
        for (int x = 0; x < 2; ++x) s[w / 8][2 * (w % 8) + x] = fmaf(s[w / 8][2 * (w % 8) + x], c, -mc);
    };
    auto raised = [&](int w) {
#pragma unroll
        for (int x = 0; x < 2; ++x) s[w / 8][2 * (w % 8) + x] = __builtin_amdgcn_exp2f(s[w / 8][2 * (w % 8) + x]);
    };
    auto summed = [&](int w) {
#pragma unroll
        for (int x = 0; x < 2; ++x) l[x] += s[w / 8][2 * (w % 8) + x];
        p[w] = at_pack(s[w / 8][2 * (w % 8)], s[w / 8][2 * (w % 8) + 1]);
    };
#pragma unroll
    for (int i = 0; i < QS; ++i) {
        __builtin_amdgcn_sched_barrier(0);
        if (i + QA < QS) kread(i + QA);
        else if (i + QA - QS < VA) vread(i + QA - QS);
        constexpr int KS = DK / 16;
        const int t = i / KS, k = i % KS;
        if (k == 0)
#pragma unroll
            for (int e = 0; e < 16; ++e) next[t][e] = 0.0f;
        next[t] = mfma32(as_bf8(ka[i]), r.q[k], next[t]);
#pragma unroll
        for (int w = QP * i; w < QP * i + QP; ++w) {
            if (w - 2 * QP >= 0 && w - 2 * QP < 16) summed(w - 2 * QP);
            if (w - QP >= 0 && w - QP < 16) raised(w - QP);
            if (w < 16) scaled(w);
        }
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int w = QP * QS; w < 16 + 2 * QP; ++w) {
        if (w - 2 * QP < 16) summed(w - 2 * QP);
        if (w - QP < 16) raised(w - QP);
    }
    r.l = l[0] + l[1];
    asm volatile("" : "+v"(r.l));   // or the sum is put off to the next tile, and with it all weights are held
    float nm = -INFINITY;
#pragma unroll
    for (int i = 0; i < VS; ++i) {
        __builtin_amdgcn_sched_barrier(0);
        if (i + VA < VS) vread(i + VA);
        const int k = i / (DV / 32), d = i % (DV / 32);
        bf8 v;
        __builtin_memcpy(&v, &va[i][0], 8);
        __builtin_memcpy(reinterpret_cast<char *>(&v) + 8, &va[i][1], 8);
        r.o[d] = mfma32(v, as_bf8(u4{p[4 * k], p[4 * k + 1], p[4 * k + 2], p[4 * k + 3]}), r.o[d]);
#pragma unroll
        for (int w = VP * i; w < VP * i + VP; ++w) nm = fmaxf(fmaxf(nm, next[w / 8][2 * (w % 8)]), next[w / 8][2 * (w % 8) + 1]);
    }
    __builtin_amdgcn_sched_barrier(0);
    mx = swap_max(nm);
}

// The same where bit j of `seen` says whether this lane's row sees key j of the tile: what it does not see takes no part,
// whatever its key and value hold. The next scores take the place of this tile's.
template <int DK, int DV>
__device__ __forceinline__ void att_tile_masked(AttRows<DK, DV> &r, v16f (&s)[2], const uint8_t *nk, const uint8_t *vt, float c,
                                                uint64_t seen, bool more)
{
    att_mask(s, seen);
    att_raise(r, att_max(s), c);
    bf8 p[4];
    att_weights(p, r, s, c);
    if (v_not_finite<DV, kAtKeys>(vt)) {
        att_values<true>(r, p, vt);
        att_not_finite<DV>(r.o, s[0], vt, 0, (uint32_t)seen);
        att_not_finite<DV>(r.o, s[1], vt, 32, (uint32_t)(seen >> 32));
    } else {
        att_values<false>(r, p, vt);
    }
    if (more) att_scores(s, r, nk);
}

}  // namespace k3moe
