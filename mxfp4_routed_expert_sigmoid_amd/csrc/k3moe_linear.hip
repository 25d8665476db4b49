// Dense products with MXFP4 matrices (k3moe_linear) and the gated pair of them
// (k3moe_glu):
//   y[t][n] = sum_k W[n][k] x[t][k],   a[t][n] = act(W1 x, W3 x)
// on bf16 or MXFP8 tokens. The format is the one of the experts (the
// "kimi-k3-in-c" README, §4 "Reduction one: the experts already ship at half a
// byte"), the activation §9's k3_situ_glu.
//
// Weights and 8-bit tokens are expanded to bf16 in registers, which is exact
// within bf16's range (an fp4 or e4m3 value times a power of two has few bits; one past
// the range is infinite, and an e4m3 value below 2^-126 that is no multiple of 2^-133,
// from a group of byte 0 to 2, loses what lies below), and multiplied on v_mfma_f32_16x16x32_bf16: exact products, fp32
// sums. (The block-scaled MFMA would take 8-bit tokens as they are at twice the rate,
// but sums each run of 16 products to about 14 bits below the largest, which shows in a
// result where large products cancel: it is not used, whatever the result's type.)
//
// Three kernels by the number of tokens, each reading every weight once per
// block of tokens that it holds:
//   k_mx_gemv    1 to 4 of at most 64 KiB together as bf16: a stream of weights,
//                bound by memory
//   k_mx_stream  more or longer ones, where tiles would not fill the card: bound by what one
//                CU's direct loads bring
//   k_mx_tile    batches: bound by the MFMAs and the expansion beside them
//
// K mapping. A 16-byte piece of a row is one block of 32 weights: in chunk c
// (128 columns) lane 16g + r of an MFMA tile holds block 4c + g of row r, and
// step s of the chunk multiplies columns 128c + 32g + 8s + [0, 8) of every g; the
// token side reads the same columns. What a chunk holds past the row's last block
// is zero on both sides: a zero weight alone would make NaN of an infinite token.
#include "k3moe_internal.h"
#include "k3moe_mx8.h"

#include <algorithm>

namespace k3moe {
namespace {

// Widest matrix: a block's rows are addressed by 32-bit offsets (256 rows x
// 2^22 / 2 bytes).
constexpr int kMaxCols = 1 << 22;
// Largest stride of token rows: a block's 128 rows are addressed by 32-bit
// offsets, 64 rows by 31-bit ones (bit 31 marks a row that is not there):
// 127 * 2^25 + 2^23 < 2^32, 63 * 2^25 + 2^23 < 2^31 bytes.
constexpr int64_t kMaxTokenStride = 1 << 24;

struct DenseParams {
    const uint8_t *w[2], *ws[2];   // packed rows [N][K / 2], scale rows [N][K / 32] (one or two matrices)
    const void *x;
    const uint8_t *xs;             // null: bf16 tokens
    void *out;
    uint8_t *outs;
    int64_t xst, xsst, ost, osst;  // row strides, elements
    int N, K, T;
    int kind;                      // k3moe_out
    int act;
    float b1, b2;
    bool vec;                      // four neighbouring results may be stored at once
};

// A dropped group (byte 255, or a block past the row's last) is cleared by
// masks, so that no lane branches: keep is 0 for it, all ones otherwise.
__device__ __forceinline__ uint32_t keep_mask(uint32_t s, uint32_t past) { return (s == 255u ? 0u : ~0u) & ~past; }
__device__ __forceinline__ u4 and_u4(u4 v, uint32_t m) { return u4{v.x & m, v.y & m, v.z & m, v.w & m}; }

// The converters' scale operand for byte s < 255: they read its exponent
// field, and a field of 0 as 2^-127.
__device__ __forceinline__ float scale_f32(uint32_t s) { return __uint_as_float(s << 23); }

// Scale bytes of a run of chunks. A load that touches 16 rows costs the address
// unit as much for four bytes of each as for 64, so the bytes of 16 chunks
// (64 of every row) are loaded at once: lane 16g + r takes bytes [16g, 16g + 16)
// of row r's run, and chunk j's dword is fetched from lane 16 (j / 4) + r when it
// is used. A run may pass the row's end (those chunks' weights are dropped),
// but not the tensor's: there the load is moved back and its bytes shifted.
// left: bytes from the run's start to the tensor's end (>= 1); total: the
// tensor's bytes.
__device__ __forceinline__ u4 run_load(const uint8_t *s, int64_t left, int64_t total, int g)
{
    u4 v = u4{0u, 0u, 0u, 0u};
    if (total < 16) {   // (a matrix or batch of fewer than 16 blocks)
        for (int i = 0; i < 16; ++i)
            if (16 * g + i < left) v[i >> 2] |= (uint32_t)s[16 * g + i] << (8 * (i & 3));
        return v;
    }
    const int64_t at = min((int64_t)(16 * g), left - 16);
    __builtin_memcpy(&v, s + at, 16);
    const int back = (int)(16 * g - at);          // bytes in front of the wanted ones; past 15: none is wanted
    if (back & 8) v = u4{v.z, v.w, 0u, 0u};
    if (back & 4) v = u4{v.y, v.z, v.w, 0u};
    const uint32_t b = 8 * (back & 3);
    return u4{__builtin_amdgcn_alignbit(v.y, v.x, b), __builtin_amdgcn_alignbit(v.z, v.y, b),
              __builtin_amdgcn_alignbit(v.w, v.z, b), v.w >> b};
}

__device__ __forceinline__ bf8 expand8_fp8(uint32_t lo, uint32_t hi, float scale)
{
    const bf2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    const bf2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    const bf2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    const bf2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    return bf8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// fp32 -> bf16, round to nearest even; NaN stays NaN.
__device__ __forceinline__ uint16_t dn_bf16(float f) { return f != f ? (uint16_t)0x7fc0u : bf16_rne(f); }

// One result (lane = row within a group of 32 rows, the token t shared by the
// 32 lanes); in: row n and token t exist. Every lane takes part.
__device__ __forceinline__ void dense_store(const DenseParams &p, int64_t t, int n, bool in, float v)
{
    if (p.kind == K3MOE_OUT_MXFP8) {
        const float m = half_wave_max(in ? mx8_mag(v) : 0.0f);
        const int s = mx8_exp(m);
        if (in) {
            static_cast<uint8_t *>(p.out)[t * p.ost + n] = (uint8_t)mx8_code(v, mx8_inv(s));
            if (n % 32 == 0) p.outs[t * p.osst + n / 32] = (uint8_t)(s + 127);
        }
    } else if (in) {
        if (p.kind == K3MOE_OUT_BF16) {
            static_cast<uint16_t *>(p.out)[t * p.ost + n] = dn_bf16(v);
        } else {
            float *o = static_cast<float *>(p.out) + t * p.ost + n;
            *o = p.kind == K3MOE_OUT_F32_ADD ? *o + v : v;
        }
    }
}

// ---------------------------------------------------------------------------
// A few tokens: the product is a stream of weights. A block owns tiles of 16
// rows of each matrix (for an MXFP8 result pairs of them, whose 32 results of a
// token share a scale); its waves split the columns, so that a narrow matrix
// still fills the card, and their fp32 sums are added in wave order. A wave
// reads 16 rows x 128 or 256 bytes per unit (U chunks) and matrix, the next unit
// in flight while one is multiplied; its share of the tokens goes into LDS
// first (behind the first weight loads), so that the loads in flight are all
// weights. A pair's two tiles are taken one after the other: side by side they
// took 173 registers and half the waves (2 x 18432 x 7168 to MXFP8: 51 us, 37 so).
//
// One token, in a graph: 1536 x 7168 5.2 us (a launch and one unit's latency),
// 7168 x 18432 16.5 us (4.3 TB/s), 2 x 18432 x 7168 33 us (4.3 TB/s); four tokens
// of 163840 x 7168 122 us (5.2 TB/s). A plain read of such sizes reaches 4 to 6.
constexpr int kGvTok = 4, kGvMaxWaves = 8;
constexpr int kGvMaxLds = 65536;   // token bytes of a block
constexpr int kGvZeros = 64;       // a block of zeros behind each token: 32 bf16 values
// A matrix of fewer tiles has a block for each (or for each pair), which the card
// schedules as they end; a longer one two blocks per CU, each with many tiles, which
// keeps the tokens in LDS and the loads in flight between them (without pairs, 512
// bytes of a row per unit instead of 256). Measured, us with a block per tile / so, on
// one token and on four (7168 columns; 2048 columns cross over earlier):
//   one matrix          700 tiles 12.0 / 13.3   15.7 / 15.7    1152 16.8 / 17.1   22.0 / 19.4
//                      1700       25.4 / 23.9   32.9 / 26.2   10240 133 / 113     171 / 124
//   one, in pairs      1152       17.2 / 19.0   20.1 / 20.7    1700 24.6 / 23.7   28.2 / 25.3
//   two                1152       33.0 / 40.1   40.1 / 43.7    1700 46.9 / 50.5   55.4 / 54.8
//                      2000       55.2 / 53.2   65.8 / 57.6    4095 103 / 96
//   two, in pairs      1152       35.8 / 46.1   40.9 / 50.3    2300 58.7 / 68.8   67.0 / 72.5
//                      3000       78.9 / 73.8   87.2 / 77.8    6000 142 / 142     157 / 147
template <int NM, bool PAIR> __host__ __device__ constexpr int gv_long() { return (1024 * NM) << PAIR; }   // tiles
constexpr int kGvBlocks = 512;

// Weights of one unit (U chunks of 128 columns) of a 16-row tile: its chunks of
// this lane's row, and the row's scale bytes of them (chunk j in dword j).
template <int U>
struct GvUnit {
    u4 a[U];
    uint32_t s[U];
};

template <int U>
__device__ __forceinline__ void gv_load(GvUnit<U> &u, const uint8_t *w, const uint8_t *s, int unit, int KB, int g)
{
    const int b0 = 4 * U * unit;
    if (b0 + 4 * U <= KB) {
#pragma unroll
        for (int j = 0; j < U; ++j) u.a[j] = *reinterpret_cast<const u4 *>(w + 16 * (b0 + 4 * j + g));
        __builtin_memcpy(u.s, s + b0, 4 * U);
    } else {  // the row's last, partial unit
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int b = b0 + 4 * j + g, bc = min(b, KB - 1);
            u.a[j] = *reinterpret_cast<const u4 *>(w + 16 * bc);
            u.s[j] = (b < KB ? (uint32_t)s[bc] : 255u) << (8 * g);
        }
    }
}

// Waits for the wave's LDS traffic, then for the block; loads into registers
// stay in flight.
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <int NM, bool X8, bool PAIR, int U>
__global__ __launch_bounds__(64 * kGvMaxWaves) void k_mx_gemv(DenseParams p, int tiles)
{
    extern __shared__ __align__(16) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nw = blockDim.x >> 6;
    const int g = lane >> 4, l16 = lane & 15;
    const int KB = p.K / 32, NU = (KB + 4 * U - 1) / (4 * U);
    const int u0 = NU * wave / nw, u1 = NU * (wave + 1) / nw;  // at least one unit each
    // this block's row tiles, one at least (without one it would not end; PAIR: an even number of them)
    tiles >>= PAIR;
    const int tile0 = (int)((int64_t)tiles * blockIdx.x / gridDim.x) << PAIR;
    const int tile1 = (int)((int64_t)tiles * (blockIdx.x + 1) / gridDim.x) << PAIR;
    const int xrow = 2 * p.K + kGvZeros;                       // LDS bytes of a token: bf16, a block of zeros
    uint8_t *xl = lds;
    float *red0 = reinterpret_cast<float *>(lds + p.T * xrow); // RB of [wave][NM][token][16]
    constexpr int RB = PAIR ? 4 : 2;
    const int rsize = nw * NM * kGvTok * 16;

    const uint8_t *wr[NM], *sr[NM];
    auto rows = [&](int tile) {
        const int64_t n = min((int64_t)16 * tile + l16, (int64_t)p.N - 1);
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            wr[m] = p.w[m] + n * (p.K / 2);
            sr[m] = p.ws[m] + n * KB;
        }
    };
    GvUnit<U> ua[NM], ub[NM];
    int lt = tile0, lu = u0;                                   // the next unit to load
    auto load = [&](GvUnit<U> (&q)[NM]) {
        if (lt >= tile1) return;
#pragma unroll
        for (int m = 0; m < NM; ++m) gv_load(q[m], wr[m], sr[m], lu, KB, g);
        if (++lu == u1) {
            lu = u0;
            rows(++lt);
        }
    };
    v4f acc[NM];
    auto clear = [&]() {
#pragma unroll
        for (int m = 0; m < NM; ++m) acc[m] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    };
    const uint8_t *bx = xl + min(l16, p.T - 1) * xrow;
    auto mul = [&](int u, const GvUnit<U> (&q)[NM]) {
        bf8 b[U][4];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int kc = min(4 * (U * u + j) + g, KB);        // past the row's last block: the zeros
#pragma unroll
            for (int s = 0; s < 4; ++s) b[j][s] = as_bf8(*reinterpret_cast<const u4 *>(bx + 64 * kc + 16 * s));
        }
        if constexpr (U == 2) __builtin_amdgcn_sched_barrier(0);   // every fragment is read before the first product
#pragma unroll
        for (int j = 0; j < U; ++j) {
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                const uint32_t sw = (q[m].s[j] >> (8 * g)) & 0xffu, keep = keep_mask(sw, 0u);
                const u4 a = and_u4(q[m].a[j], keep);
                const float f = scale_f32(sw & keep);
#pragma unroll
                for (int s = 0; s < 4; ++s) acc[m] = mfma_bf16(dequant8_bf16(a[s], f), b[j][s], acc[m]);
            }
        }
    };
    // A tile's sums go to LDS; they are added in wave order, one value per thread: 16 rows of a token, or the 32 of
    // a pair behind its second tile (an MXFP8 group). The areas take turns, so that a wave may be one tile (pair)
    // ahead of those that still add.
    auto finish = [&](int tile) {
        const int area = (tile - tile0) & (RB - 1);
        float *red = red0 + area * rsize;
        if (l16 < p.T) {
#pragma unroll
            for (int m = 0; m < NM; ++m)
                *reinterpret_cast<float4 *>(red + ((wave * NM + m) * kGvTok + l16) * 16 + 4 * g) =
                    float4{acc[m][0], acc[m][1], acc[m][2], acc[m][3]};
        }
        clear();
        if (PAIR && !(area & 1)) return;
        lds_barrier();
        constexpr int ROWS = PAIR ? 32 : 16;
        if constexpr (PAIR) red -= rsize;                      // the pair's first tile
        const int n0 = 16 * (tile - PAIR);
        for (int i = tid; i < ROWS * ((p.T + 1) & ~1); i += 64 * nw) {
            const int row = i % ROWS, tok = i / ROWS, tc = min(tok, p.T - 1), n = n0 + row;
            const float *from = red + (row >> 4) * rsize + tc * 16 + (row & 15);
            float v[NM];
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                v[m] = 0.0f;
                for (int w = 0; w < nw; ++w) v[m] += from[(w * NM + m) * kGvTok * 16];
            }
            float y = v[0];
            if constexpr (NM == 2) y = act_fn(v[0], v[1], p.act, p.b1, p.b2);
            dense_store(p, tok, n, tok < p.T && row < p.N - n0, y);
        }
    };

    rows(tile0);
    load(ua);
    clear();
    {
        // the wave's columns of every token, as bf16, 16 bytes at a time (eight in flight per lane took 1 to 2 % longer)
        const int c0 = 128 * U * u0, per = (min(128 * U * u1, p.K) - c0) / (X8 ? 16 : 8);   // 16-byte pieces of a token
        for (int i = lane; i < p.T * per; i += 64) {
            const int t = i / per, c = c0 + (X8 ? 16 : 8) * (i - t * per);
            const u4 x = *reinterpret_cast<const u4 *>(static_cast<const uint8_t *>(p.x) + (t * p.xst + c) * (X8 ? 1 : 2));
            uint8_t *at = xl + t * xrow + 2 * c;
            if constexpr (X8) {
                const uint32_t sx = p.xs[t * p.xsst + c / 32], keep = keep_mask(sx, 0u);
                const u4 v = and_u4(x, keep);
                const float f = scale_f32(sx & keep);
                bf8 *d = reinterpret_cast<bf8 *>(at);
                d[0] = expand8_fp8(v.x, v.y, f), d[1] = expand8_fp8(v.z, v.w, f);
            } else {
                *reinterpret_cast<u4 *>(at) = x;
            }
        }
        if (__builtin_expect(KB % (4 * U) != 0, 0) && lane < 4 * p.T)
            *reinterpret_cast<u4 *>(xl + (lane >> 2) * xrow + 2 * p.K + 16 * (lane & 3)) = u4{0u, 0u, 0u, 0u};
        wave_lds_sync();
    }
    // two units at a time: while one is multiplied the other is in flight, across the tiles' borders
    int t = tile0, u = u0;
    auto next = [&]() {
        if (++u == u1) {
            finish(t);
            u = u0;
            ++t;
        }
    };
    for (;;) {
        load(ub);
        mul(u, ua);
        next();
        if (t == tile1) break;
        load(ua);
        mul(u, ub);
        next();
        if (t == tile1) break;
    }
}

// ---------------------------------------------------------------------------
typedef __attribute__((address_space(3))) void lds_void;

#ifdef __HIP_DEVICE_COMPILE__
// A buffer resource over the 4 GiB behind p: the direct loads take 32-bit
// offsets from it (and, unlike those of the global form, leave the waits for
// loads into registers exact).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buf_src(const uint8_t *p, int bytes = -1)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(p), 0, bytes, 0x00020000);
}
#endif

// Waits until at most N of the wave's memory loads are in flight and its LDS
// traffic is done, then for the block.
template <int N>
__device__ __forceinline__ void tile_barrier()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// ---------------------------------------------------------------------------
// More tokens on a card that tiles would not fill. A block owns 32 rows of
// each matrix and 16 NT tokens; each of its eight waves takes one of the two
// row tiles and every fourth part of the columns, four chunks of 128 columns (a
// phase) at a time, and the four parts' sums are added at the end in their
// order. The tokens of a phase go into LDS by direct loads of whole rows, and
// so do each wave's weights, four lanes to a row: read from memory in operand
// order, a load costs the address unit about a cycle per lane.
//
// Measured on 7168 rows x 7168, in a graph: 8 MXFP8 tokens 10.4 us, 8 bf16
// tokens 10.6, 48 MXFP8 tokens 18.7 (264 TFLOP/s), 48 bf16 tokens 18.6. No unit of
// the card is busy for much more than half of that (data return of the loads 44 to 53 %,
// MFMAs 7 to 12 %, L2 misses only the weights): two waves per SIMD wait 45 % of
// their cycles for loads and barriers. Every block reads its tokens anew (and
// expands those in 8 bits), which only more rows per block would change, and those
// would leave CUs idle. Phases of eight chunks,
// one per wave and both row tiles, do not hold 64 bf16 tokens (301 tokens x 1001 x
// 2080: 16.0 us, 9.1 so).
//
// LDS holds slot j (16 bytes) of token row r at slot j ^ (r & 15).
constexpr int kStW = 8, kStC = 4;                 // waves, chunks of a phase
constexpr int kStMaxBuf = 3;                      // (8 MXFP8 tokens x 7168 x 7168: 10.6 us, 11.0 with four buffers, 11.6 with six)
template <bool X8> __host__ __device__ constexpr int st_es() { return X8 ? 1 : 2; }  // bytes per token element
constexpr int kMaxLds = 163840;
// An offset behind every token's (63 * 2^25 + 2^23 at most): read as zeros.
constexpr int kStOut = 0x7f000000;
template <int NM, bool X8, int NT> __host__ __device__ constexpr int st_x() { return 16 * NT * 128 * kStC * st_es<X8>(); }   // tokens of a phase
template <int NM, bool X8, int NT> __host__ __device__ constexpr int st_buf() { return st_x<NM, X8, NT>() + kStW * NM * 1024; }
template <int NM, bool X8, int NT> __host__ __device__ constexpr int st_nbuf()
{
    constexpr int n = kMaxLds / st_buf<NM, X8, NT>();
    return n > kStMaxBuf ? kStMaxBuf : n;
}
template <int NM, bool X8, int NT> __host__ __device__ constexpr int st_lds()
{
    constexpr int x = st_nbuf<NM, X8, NT>() * st_buf<NM, X8, NT>(), red = kStW * NM * NT * 1024;
    static_assert(x <= kMaxLds && red <= kMaxLds && st_nbuf<NM, X8, NT>() >= 2, "a block's LDS");
    return x > red ? x : red;
}

template <int NM, bool X8, int NT>
__global__ __launch_bounds__(64 * kStW) void k_mx_stream(DenseParams p, int tok_blocks)
{
#ifdef __HIP_DEVICE_COMPILE__   // the buffer resource type exists on the device side only
    constexpr int ES = st_es<X8>(), XBUF = st_x<NM, X8, NT>(), BUF = st_buf<NM, X8, NT>(), NB = st_nbuf<NM, X8, NT>(), D = NB - 1;
    constexpr int XL = NT * ES;                   // direct loads per wave and phase
    extern __shared__ __align__(16) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, l16 = lane & 15;
    const int uw = __builtin_amdgcn_readfirstlane(wave);
    // block b runs on XCD b mod 8: each XCD takes one run of blocks, those of the same rows next to each other
    const int nt = gridDim.x, xcd = blockIdx.x & 7, per = nt >> 3, rest = nt & 7;
    const int at = xcd * per + min(xcd, rest) + (int)(blockIdx.x >> 3);
    const int rb = at / tok_blocks, tb = at - rb * tok_blocks;
    const int n0 = 32 * rb, t0 = 16 * NT * tb;
    const int KB = p.K / 32, NC = (KB + 3) / 4, NP = (NC + kStC - 1) / kStC;   // chunks, phases
    // a wave multiplies one of the two row tiles by the chunks [c0(s), c0(s + 1)) of its slot s, one per phase
    auto c0 = [&](int s) { return NC * s / kStC; };
    const int cs = wave & (kStC - 1), rt = wave >> 2;
    const int cw = c0(cs), cn = c0(cs + 1) - cw;
    // Weights, four lanes per row (a lane of the MFMA's order per row would cost the address unit a cycle per
    // lane): a load brings 16 bytes x 4 of the wave's 16 rows, slot j of row r at j ^ (r / 4 mod 4).
    const uint8_t *sr[NM];
    __amdgpu_buffer_rsrc_t wsrc[NM];
    int64_t xleft[NT];
    const int64_t ns = min(n0 + 16 * rt + l16, p.N - 1), sleft = (p.N - ns) * KB;
    const uint32_t wo = (uint32_t)min(16 * rt + (lane >> 2), p.N - 1 - n0) * (uint32_t)(p.K / 2);
#pragma unroll
    for (int m = 0; m < NM; ++m) {
        wsrc[m] = buf_src(p.w[m] + (size_t)n0 * (p.K / 2));
        sr[m] = p.ws[m] + ns * KB;
    }
    const int wj = (lane & 3) ^ (lane >> 4);      // this lane's block of a chunk
    const uint8_t *xsr[NT];
    if constexpr (X8) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int64_t tt = min(t0 + 16 * t + l16, p.T - 1);
            xsr[t] = p.xs + tt * p.xsst;
            xleft[t] = (p.T - 1 - tt) * p.xsst + KB;
        }
    }
    auto wload = [&](int ph, int buf) {
        const int kc = min(4 * (cw + max(min(ph, cn - 1), 0)) + wj, KB - 1);   // (a wave may have no chunk)
#pragma unroll
        for (int m = 0; m < NM; ++m)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(wsrc[m], (lds_void *)(lds + buf * BUF + XBUF + (uw * NM + m) * 1024), 16,
                                                     (int)(wo + 16u * (uint32_t)kc), 0, 0, 0);
        asm volatile("" ::: "memory");            // no load moves behind the products
    };
    struct Scales {                               // of 16 phases
        u4 w[NM], x[X8 ? NT : 1];
    };
    auto sload = [&](int seg, Scales &q) {
        const int o = 4 * min(cw + 16 * seg, (KB - 1) / 4);
#pragma unroll
        for (int m = 0; m < NM; ++m) q.w[m] = run_load(sr[m] + o, sleft - o, (int64_t)p.N * KB, g);
        if constexpr (X8) {
#pragma unroll
            for (int t = 0; t < NT; ++t) q.x[t] = run_load(xsr[t] + o, xleft[t] - o, (p.T - 1) * p.xsst + KB, g);
        }
    };
    // direct loads: 64 slots per wave and load, one row of bf16 tokens or two of 8-bit ones, of all four chunks
    constexpr int RL = 2 / ES, SL = 64 / RL;      // rows per load, slots per row
    const __amdgpu_buffer_rsrc_t xsrc = buf_src(static_cast<const uint8_t *>(p.x) + (int64_t)t0 * p.xst * ES, kStOut);
    uint32_t xo[XL];                              // row offsets; rows past the last token lie outside, read as zeros
    int xs0[ES], xend[ES];                        // this lane's slot of phase 0 (rows 8 apart take turns in bf16), its run's end
#pragma unroll
    for (int i = 0; i < XL; ++i) {
        const int row = RL * (kStW * i + uw) + (RL == 1 ? 0 : lane >> 5);
        xo[i] = t0 + row < p.T ? (uint32_t)row * (uint32_t)(p.xst * ES) : 0x80000000u;
        const int j = (lane & (SL - 1)) ^ (row & 15), w = j / (8 * ES);   // its slot of the phase, its chunk's
        if (i < ES) xs0[i] = 8 * ES * c0(w) + (j & (8 * ES - 1)), xend[i] = min(8 * ES * c0(w + 1), p.K * ES / 16);
    }
    auto xload = [&](int ph, int buf) {
        uint32_t slot[ES];
#pragma unroll
        for (int i = 0; i < ES; ++i) {
            const int j = xs0[i] + 8 * ES * ph;
            if constexpr (X8) slot[i] = 16u * (uint32_t)min(j, p.K / 16 - 1);   // (dropped by their scale bytes, below)
            else slot[i] = j < xend[i] ? 16u * (uint32_t)j : (uint32_t)kStOut;  // past its run: outside, zeros
        }
#pragma unroll
        for (int i = 0; i < XL; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(xsrc, (lds_void *)(lds + buf * BUF + 1024 * (kStW * i + uw)), 16,
                                                     (int)(xo[i] + slot[i % ES]), 0, 0, 0);
        asm volatile("" ::: "memory");            // no load moves behind the products
    };
    v4f acc[NM][NT];
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[m][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    // phase ph = 16 seg + 4 quarter + k with the scales of its segment
    auto mul = [&](int ph, int quarter, int k, const Scales &sc, int buf) {
        const uint32_t past = 4 * (cw + ph) + g < KB && ph < cn ? 0u : ~0u;   // no block of this wave: zeros
        const uint8_t *B = lds + buf * BUF + l16 * 512 * ES;
        const uint8_t *A = lds + buf * BUF + XBUF + wave * NM * 1024 + 64 * l16 + 16 * (g ^ (l16 >> 2));
        const int from = 16 * quarter + l16;      // the lane that holds the phase's scales
        u4 a[NM];
        uint32_t sw[NM], xsb[NT];
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            const uint32_t sv = ((uint32_t)__shfl((int)sc.w[m][k], from) >> (8 * g)) & 0xffu, keep = keep_mask(sv, past);
            a[m] = and_u4(*reinterpret_cast<const u4 *>(A + m * 1024), keep);
            sw[m] = sv & keep;
        }
        if constexpr (X8) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {   // (every lane takes part in the exchange)
                const uint32_t sx = ((uint32_t)__shfl((int)sc.x[t][k], from) >> (8 * g)) & 0xffu;
                xsb[t] = (sx & ~past) | (255u & past);   // past the last block: dropped
            }
        }
        // every fragment of the chunk is read before the first product (the compiler would read each where it
        // is used, a wait of the LDS's latency every few MFMAs)
        constexpr int XF = X8 ? 2 : 4;
        u4 x[NT][XF];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < XF; ++i) {
                const int slot = 8 * ES * cs + 2 * ES * g + i;
                x[t][i] = *reinterpret_cast<const u4 *>(B + 8192 * ES * t + 16 * (slot ^ l16));
            }
        __builtin_amdgcn_sched_barrier(0);
        float xf[NT];
        if constexpr (X8) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const uint32_t keep = keep_mask(xsb[t], 0u);
                x[t][0] = and_u4(x[t][0], keep), x[t][1] = and_u4(x[t][1], keep);
                xf[t] = scale_f32(xsb[t] & keep);
            }
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            bf8 w[NM];
#pragma unroll
            for (int m = 0; m < NM; ++m) w[m] = dequant8_bf16(a[m][s], scale_f32(sw[m]));
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                bf8 b;
                if constexpr (X8) b = expand8_fp8(x[t][s >> 1][2 * (s & 1)], x[t][s >> 1][2 * (s & 1) + 1], xf[t]);
                else b = as_bf8(x[t][s]);
#pragma unroll
                for (int m = 0; m < NM; ++m) acc[m][t] = mfma_bf16(w[m], b, acc[m][t]);
            }
        }
    };

    // Pipeline. A phase's tokens and weights are loaded D phases ahead; phase ph
    // waits until only the loads of the D - 1 phases behind it are in flight,
    // and for the block. A buffer is loaded again behind the barrier that
    // follows the phase which read it. A wave's phases past
    // its last chunk load that again and are not multiplied.
    constexpr int LPP = XL + NM;                  // loads per phase
    Scales sc;
    sload(0, sc);
#pragma unroll
    for (int k = 0; k < D; ++k) {
        wload(k, k);
        xload(min(k, NP - 1), k);
    }
    int cur = 0, in = D;
    for (int ph = 0; ph < NP; ph += 4) {
        if (ph > 0 && ph % 16 == 0) sload(ph / 16, sc);
        static_for<0, 4>([&](auto kk) {
            constexpr int k = decltype(kk)::value;
            if (ph + k < NP) {
                tile_barrier<LPP *(D - 1)>();
                wload(ph + k + D, in);
                xload(min(ph + k + D, NP - 1), in);
                mul(ph + k, (ph >> 2) & 3, k, sc, cur);
                cur = cur == NB - 1 ? 0 : cur + 1;
                in = in == NB - 1 ? 0 : in + 1;
            }
        });
    }
    tile_barrier<0>();   // the buffers become the sums' area

    // the four chunk slots' sums are added in their order
    float4 *red = reinterpret_cast<float4 *>(lds);
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)              // [token][row]: lane l16 holds rows 4g + i of token l16
            red[((wave * NM + m) * NT + t) * 64 + 4 * l16 + g] =
                float4{acc[m][t][0], acc[m][t][1], acc[m][t][2], acc[m][t][3]};
    tile_barrier<0>();
#pragma unroll
    for (int q = 0; q < NT; ++q) {
        const int tok = tid >> 5, row = tid & 31, t = t0 + 16 * q + tok;
        float v[NM];
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            v[m] = 0.0f;
#pragma unroll
            for (int w = 0; w < kStC; ++w)
                v[m] += reinterpret_cast<const float *>(red + (((w + kStC * (row >> 4)) * NM + m) * NT + q) * 64)[16 * tok + (row & 15)];
        }
        float y = v[0];
        if constexpr (NM == 2) y = act_fn(v[0], v[1], p.act, p.b1, p.b2);
        dense_store(p, t, n0 + row, t < p.T && n0 + row < p.N, y);
    }
#endif
}

// ---------------------------------------------------------------------------
// Tiles for batches. A block of 8 waves owns 256 weight rows (256 of the one
// matrix, or 128 of each of the two) and 128 tokens; a wave 64 rows x 64
// tokens (gate and up rows of the same columns, so the activation stays in
// its lanes). Tokens and packed weights pass through LDS, 128 columns per step,
// by direct loads into three buffers (four of the smaller MXFP8 steps), one
// barrier per step; 8-bit tokens that are expanded go through registers, once
// per block instead of once per wave. Rows rather than tokens are the long
// side because a token's bytes are four times a weight row's: LDS reads take
// half the cycles of the MFMAs.
//
// 2048 tokens x 7168 x 18432: bf16 to bf16 508 us (1.07 PFLOP/s; the library's
// bf16 product of that size 522), MXFP8 to bf16 557 us (0.97: the expansion of the
// tokens), += 577. MFMAs are busy for 43 and 39 % of it. Of 514 us for bf16, 349 were left
// without loads and LDS reads, the MFMAs with the expansion of the weights, and 388
// with the reads; 448 tiles on 256 CUs are two rounds of which the second is 3/4 full.
//
// LDS holds slot j (16 bytes) of token row r at slot j ^ (r & 15), so a
// fragment read (one slot of 16 rows) touches every bank once.
constexpr int kTlRows = 256, kTlTok = 128, kTlWaves = 8;
// An offset behind every token's (127 * 2^25 + 2^23 at most): read as zeros.
constexpr int kTlOut = (int)0xff000000u;
// Four neighbouring results (columns n .. n + 3 of token t; the 8 lanes of an
// octet hold one group of 32 columns). nin: how many of them exist (0: none).
__device__ __forceinline__ void dense_store4(const DenseParams &p, int64_t t, int n, int nin, float4 y)
{
    const float v[4] = {y.x, y.y, y.z, y.w};
    if (p.kind == K3MOE_OUT_MXFP8) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = fmaxf(m, i < nin ? mx8_mag(v[i]) : 0.0f);
        m = octet_max(m);
        const int s = mx8_exp(m);
        const float inv = mx8_inv(s);
        uint8_t *o = static_cast<uint8_t *>(p.out) + t * p.ost + n;
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = mx8_code(v[i], inv);
        if (nin == 4 && p.vec) {
            *reinterpret_cast<uint32_t *>(o) = c[0] | (c[1] << 8) | (c[2] << 16) | (c[3] << 24);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < nin) o[i] = (uint8_t)c[i];
        }
        if (nin > 0 && n % 32 == 0) p.outs[t * p.osst + n / 32] = (uint8_t)(s + 127);
    } else if (p.kind == K3MOE_OUT_BF16) {
        uint16_t *o = static_cast<uint16_t *>(p.out) + t * p.ost + n;
        if (nin == 4 && p.vec) {
            *reinterpret_cast<uint2 *>(o) = uint2{(uint32_t)dn_bf16(v[0]) | ((uint32_t)dn_bf16(v[1]) << 16),
                                                  (uint32_t)dn_bf16(v[2]) | ((uint32_t)dn_bf16(v[3]) << 16)};
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < nin) o[i] = dn_bf16(v[i]);
        }
    } else {
        float *o = static_cast<float *>(p.out) + t * p.ost + n;
        const bool add = p.kind == K3MOE_OUT_F32_ADD;
        if (nin == 4 && p.vec) {
            float4 z = add ? *reinterpret_cast<const float4 *>(o) : float4{0.0f, 0.0f, 0.0f, 0.0f};
            z.x += y.x, z.y += y.y, z.z += y.z, z.w += y.w;
            *reinterpret_cast<float4 *>(o) = z;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < nin) o[i] = add ? o[i] + v[i] : v[i];
        }
    }
}

// A step is 128 columns: 64 bytes of every weight row, 256 (as bf16) of every
// token, one dword of every scale row. The buffers of a block:
constexpr int kTlBufs = 3, kTlXRow = 256;
constexpr int kTlWBuf = kTlRows * 64, kTlSRows = 64 * kTlWaves;  // one scale dword per thread
constexpr int kTlBuf = kTlTok * kTlXRow + kTlWBuf + 4 * kTlSRows, kTlLds = kTlBufs * kTlBuf;

// LDS stores of the tile pipeline. As plain stores the compiler would first
// wait for every direct load in flight, which may write the same LDS for all
// it knows; tile_barrier waits for them. (The LDS address is the low half of
// a shared pointer.)
__device__ __forceinline__ void lds_put(const uint8_t *at, uint32_t v)
{
    asm volatile("ds_write_b32 %0, %1" ::"v"((uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t *)at), "v"(v)
                 : "memory");
}
__device__ __forceinline__ void lds_put16(const uint8_t *at, bf8 v)
{
    asm volatile("ds_write_b128 %0, %1" ::"v"((uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t *)at), "v"(v)
                 : "memory");
}

template <int NM, bool X8>
__global__ __launch_bounds__(64 * kTlWaves) void k_mx_tile(DenseParams p, int tok_tiles)
{
#ifdef __HIP_DEVICE_COMPILE__   // the buffer resource type exists on the device side only
    constexpr int NB = kTlBufs, BUF = kTlBuf, XR = kTlXRow;
    constexpr int XB = kTlTok * XR;               // a buffer: tokens, weights, scales
    extern __shared__ __align__(16) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, l16 = lane & 15;
    const int wn = wave >> 1, wt = wave & 1;
    // Neighbouring blocks run on different XCDs (block b on b mod 8): each XCD takes one run of tiles, in an
    // order that goes through four token tiles for every row block, so that the tiles in flight in it share
    // weights and tokens in its L2 (2048 x 7168 x 18432 bf16: 513 us, token tiles in order 523)
    const int nt = gridDim.x, xcd = blockIdx.x & 7, per = nt >> 3, rest = nt & 7;
    const int tile = xcd * per + min(xcd, rest) + (int)(blockIdx.x >> 3);
    const int group = tile / (nt / tok_tiles * 4), gt0 = 4 * group, gt = min(4, tok_tiles - gt0);
    const int in_group = tile - nt / tok_tiles * gt0, rb = in_group / gt, tb = gt0 + in_group - rb * gt;
    const int n0 = rb * (kTlRows / NM), t0 = tb * kTlTok;
    const int KB = p.K / 32, NS = (KB + 3) / 4;

    // Weight staging: LDS row i < 256 / NM holds row n0 + i of the first matrix, the others the second's.
    // Four threads per row, two passes; offsets from the block's first row fit 32 bits.
    auto lrow = [&](int i) { return NM == 1 ? i : i & (kTlRows / 2 - 1); };
    uint32_t wo[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) wo[i] = (uint32_t)min(lrow((tid >> 2) + 128 * i), p.N - 1 - n0) * (uint32_t)(p.K / 2);
    __amdgpu_buffer_rsrc_t wsrc[NM];
#pragma unroll
    for (int m = 0; m < NM; ++m) wsrc[m] = buf_src(p.w[m] + (size_t)n0 * (p.K / 2));
    const int wj = (tid & 3) ^ ((tid >> 4) & 3);  // slot j of row r lies at j ^ (r / 4 mod 4)
    auto wdirect = [&](int k, int buf) {
        const uint32_t kc = 16u * (uint32_t)min(4 * k + wj, KB - 1);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(wsrc[NM == 1 ? 0 : i],
                                                     (lds_void *)(lds + buf * BUF + XB + (512 * i + 64 * wave) * 16), 16,
                                                     (int)(wo[i] + kc), 0, 0, 0);
    };
    // Scales: thread i < 256 holds the dword (four blocks) of LDS weight row i in a register for a step before it
    // goes to its buffer (the other threads a copy: every wave issues the same loads); blocks past the row's last
    // read as 255. K >= 128: the last dword of a row is loaded and shifted.
    const uint8_t *sp = p.ws[NM == 1 ? 0 : (tid & 255) >> 7] + (size_t)min(n0 + lrow(tid & 255), p.N - 1) * KB;
    uint32_t sreg = 0;
    auto sload = [&](int k) { __builtin_memcpy(&sreg, sp + min(4 * k, KB - 4), 4); };
    auto sstore = [&](int k, int buf) {
        const int sh = 8 * max(0, 4 * k + 4 - KB);   // blocks past the last: 0, or 8 to 24 bits
        lds_put(lds + buf * BUF + XB + kTlWBuf + 4 * tid, (sreg >> sh) | ~(~0u >> sh));
    };

    // Token staging. bf16: direct, slots of 16 bytes, XP per thread. MXFP8: two slots of 16 values per thread, held
    // in registers for a step and expanded on their way into LDS.
    constexpr int ES = X8 ? 1 : 2;                // bytes per token element in memory
    constexpr int SL = XR / 16, XP = XB / 8192;   // slots per row, passes
    constexpr int EP = 2;
    const uint8_t *xb = static_cast<const uint8_t *>(p.x);
    const uint8_t *xr[EP], *xsr[EP];
    uint32_t xo[XP];
    const __amdgpu_buffer_rsrc_t xsrc = buf_src(xb + (int64_t)t0 * p.xst * ES, kTlOut);
    if constexpr (X8) {
#pragma unroll
        for (int i = 0; i < EP; ++i) {
            const int64_t t = min(t0 + (tid >> 3) + 64 * i, p.T - 1);
            xr[i] = xb + t * p.xst;
            xsr[i] = p.xs + t * p.xsst;
        }
    } else {
#pragma unroll
        for (int i = 0; i < XP; ++i)
            xo[i] = (uint32_t)min((tid + 512 * i) / SL, p.T - 1 - t0) * (uint32_t)(p.xst * ES);
    }
    const int last = p.K * ES / 16 - 1;           // last slot of a token row
    const int xsw = (tid >> 4) & 15;              // slot j of token r lies at j ^ (r mod 16) (the passes keep r mod 16)
    auto xdirect = [&](int k, int buf) {
        const int slot = SL * k + ((tid & (SL - 1)) ^ xsw);
#pragma unroll
        for (int i = 0; i < XP; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(xsrc, (lds_void *)(lds + buf * BUF + (512 * i + 64 * wave) * 16), 16,
                                                     (int)(slot <= last ? xo[i] + 16u * (uint32_t)slot : (uint32_t)kTlOut), 0, 0, 0);
    };
    u4 xe[EP];
    uint32_t xes[EP];
    auto eload = [&](int k) {
        const int slot = min(8 * k + (tid & 7), last);
#pragma unroll
        for (int i = 0; i < EP; ++i) {
            xe[i] = *reinterpret_cast<const u4 *>(xr[i] + 16 * (int64_t)slot);
            xes[i] = xsr[i][slot >> 1];
        }
    };
    auto estore = [&](int k, int buf) {
#pragma unroll
        for (int i = 0; i < EP; ++i) {
            const int row = (tid >> 3) + 64 * i, j = 2 * (tid & 7);
            const uint32_t keep = keep_mask(xes[i], 0u);
            const float f = scale_f32(xes[i] & keep);
            const u4 v = and_u4(xe[i], keep);
            uint8_t *d = lds + buf * BUF + row * 256;
            lds_put16(d + 16 * (j ^ (row & 15)), expand8_fp8(v.x, v.y, f));
            lds_put16(d + 16 * ((j + 1) ^ (row & 15)), expand8_fp8(v.z, v.w, f));
        }
        if (4 * k + 4 > KB && 8 * k + (tid & 7) > last) {   // behind the row's last slot: zeros
#pragma unroll
            for (int i = 0; i < EP; ++i) {
                const int row = (tid >> 3) + 64 * i, j = 2 * (tid & 7);
                uint8_t *d = lds + buf * BUF + row * 256;
                lds_put16(d + 16 * (j ^ (row & 15)), bf8{});
                lds_put16(d + 16 * ((j + 1) ^ (row & 15)), bf8{});
            }
        }
    };

    v4f acc[4][4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[r][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    // this wave's four row tiles: LDS rows 64 wn + 16 r, or 32 wn + 16 (r mod 2) of either matrix's half
    int arow[4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
        arow[r] = (NM == 1 ? 64 * wn + 16 * r : 128 * (r >> 1) + 32 * wn + 16 * (r & 1)) + l16;
    const int asl = 16 * (g ^ (l16 >> 2));        // this lane's slot of them

    auto compute = [&](int buf) {
        const uint8_t *B = lds + buf * BUF + (64 * wt + l16) * XR;
        const uint8_t *A = lds + buf * BUF + XB, *S = A + kTlWBuf;
        u4 a[4];
        uint32_t s4[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            a[r] = *reinterpret_cast<const u4 *>(A + arow[r] * 64 + asl);
            s4[r] = *reinterpret_cast<const uint32_t *>(S + 4 * arow[r]);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const uint32_t sv = (s4[r] >> (8 * g)) & 0xffu, keep = keep_mask(sv, 0u);
            a[r] = and_u4(a[r], keep);
            s4[r] = sv & keep;
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            bf8 b[4];
#pragma unroll
            for (int t = 0; t < 4; ++t)
                b[t] = as_bf8(*reinterpret_cast<const u4 *>(B + 16 * XR * t + 16 * ((4 * g + s) ^ l16)));
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const bf8 av = dequant8_bf16(a[r][s], scale_f32(s4[r]));
#pragma unroll
                for (int t = 0; t < 4; ++t) acc[r][t] = mfma_bf16(av, b[t], acc[r][t]);
            }
        }
    };

    // Pipeline. The loads of step k are issued in step k - NB + 1: first those
    // through registers (stored to their buffer one step later), then the
    // direct ones. Step k waits until only the loads of the NB - 2 steps
    // behind it are in flight, and for the block; its buffer is then whole,
    // and the buffer of step k - 1 is read and free for step k + NB - 1. Steps
    // past the last load the last one's operands again, so that every step
    // issues LPS loads (from empty buffers, whose descriptors are then made
    // anew for each step, the kernel took 2 to 7 % longer).
    constexpr int LPS = 1 + (X8 ? 2 * EP : XP) + 2;
    constexpr int D = NB - 1;
    auto issue = [&](int k, int buf) {
        const int kc = min(k, NS - 1);
        sload(kc);
        if constexpr (X8) eload(kc);
        wdirect(kc, buf);
        if constexpr (!X8) xdirect(kc, buf);
        asm volatile("" ::: "memory");            // no load moves behind the products
    };
    auto settle = [&](int k, int buf) {
        sstore(min(k, NS - 1), buf);
        if constexpr (X8) estore(min(k, NS - 1), buf);
    };
#pragma unroll
    for (int k = 0; k < D; ++k) {
        issue(k, k);
        if (k < D - 1) settle(k, k);
    }
    int cur = 0, in = D;                          // buffers of step k and of step k + D
    for (int k = 0; k < NS; ++k) {
        // the newest loads in registers (step k + D - 1) go to their buffer, then step k's operands are awaited
        const int prev = in == 0 ? NB - 1 : in - 1;
        settle(k + D - 1, prev);
        tile_barrier<LPS *(D - 1)>();
        issue(k + D, in);
        compute(cur);
        cur = cur == NB - 1 ? 0 : cur + 1;
        in = in == NB - 1 ? 0 : in + 1;
    }
    tile_barrier<0>();  // the buffers become the waves' transpose areas

    // Epilogue, 16 tokens at a time: [token][row] through the wave's own LDS, then four
    // neighbouring columns per lane (16 lanes: 64 rows of one matrix, or the first 8 of them
    // 32 activations).
    float *tr = reinterpret_cast<float *>(lds) + wave * (16 * 68);
    constexpr int CT = 64 / NM;                    // columns per wave
    constexpr int LPT = CT / 4, TPP = 64 / LPT;    // lanes per token, tokens per pass
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int r = 0; r < 4 / NM; ++r) {
            float4 v;
            if constexpr (NM == 1) {
                v = float4{acc[r][t][0], acc[r][t][1], acc[r][t][2], acc[r][t][3]};
            } else {
                v = float4{act_fn(acc[r][t][0], acc[r + 2][t][0], p.act, p.b1, p.b2),
                           act_fn(acc[r][t][1], acc[r + 2][t][1], p.act, p.b1, p.b2),
                           act_fn(acc[r][t][2], acc[r + 2][t][2], p.act, p.b1, p.b2),
                           act_fn(acc[r][t][3], acc[r + 2][t][3], p.act, p.b1, p.b2)};
            }
            *reinterpret_cast<float4 *>(tr + 68 * l16 + 16 * r + 4 * g) = v;
        }
        wave_lds_sync();
#pragma unroll
        for (int q = 0; q < 16 / TPP; ++q) {
            const int tok = q * TPP + lane / LPT, col = 4 * (lane % LPT);
            const float4 v = *reinterpret_cast<const float4 *>(tr + 68 * tok + col);
            const int tt = t0 + 64 * wt + 16 * t + tok, n = n0 + CT * wn + col;
            dense_store4(p, tt, n, tt < p.T ? max(0, min(4, p.N - n)) : 0, v);
        }
        wave_lds_sync();
    }
#endif
}

// work-items of a launch are counted in 32 bits
constexpr int64_t kMaxItems = ((int64_t)1 << 32) - 1;

template <int NM, bool X8>
void launch_tile(const DenseParams &p, int64_t blocks, int tok_tiles, hipStream_t s)
{
    (void)hipFuncSetAttribute(reinterpret_cast<const void *>(&k_mx_tile<NM, X8>),
                              hipFuncAttributeMaxDynamicSharedMemorySize, kTlLds);
    k_mx_tile<NM, X8><<<(unsigned)blocks, 64 * kTlWaves, kTlLds, s>>>(p, tok_tiles);
}

template <int NM, bool X8, bool PAIR, int U>
void launch_gemv(const DenseParams &p, int tiles, int blocks, hipStream_t s)
{
    blocks = std::min(blocks, tiles >> PAIR);   // each has a tile
    const int NU = (p.K / 32 + 4 * U - 1) / (4 * U);
    // waves per block: the fewest that give the same longest share as the most
    const int share = (NU + kGvMaxWaves - 1) / kGvMaxWaves, nw = (NU + share - 1) / share;
    const int lds = p.T * (2 * p.K + kGvZeros) + (PAIR ? 4 : 2) * nw * NM * kGvTok * 64;
    if (lds > 65536)
        (void)hipFuncSetAttribute(reinterpret_cast<const void *>(&k_mx_gemv<NM, X8, PAIR, U>),
                                  hipFuncAttributeMaxDynamicSharedMemorySize, kGvMaxLds + 65536);
    k_mx_gemv<NM, X8, PAIR, U><<<(unsigned)blocks, 64 * nw, lds, s>>>(p, tiles);
}

template <int NM, bool X8, int NT>
k3moe_status launch_stream(const DenseParams &p, hipStream_t s)
{
    const int64_t rb = ((int64_t)p.N + 31) / 32, tb = ((int64_t)p.T + 16 * NT - 1) / (16 * NT);
    if (rb * tb > kMaxItems / (64 * kStW)) return K3MOE_E_UNSUPPORTED_SHAPE;
    if (st_lds<NM, X8, NT>() > 65536)
        (void)hipFuncSetAttribute(reinterpret_cast<const void *>(&k_mx_stream<NM, X8, NT>),
                                  hipFuncAttributeMaxDynamicSharedMemorySize, st_lds<NM, X8, NT>());
    k_mx_stream<NM, X8, NT><<<(unsigned)(rb * tb), 64 * kStW, st_lds<NM, X8, NT>(), s>>>(p, (int)tb);
    return K3MOE_OK;
}

// Time models (us) that choose between the batch kernels and the streaming
// kernel's tokens per block, from what they measured at 8 to 2048 tokens x 512 to
// 18432 rows x 2048 and 7168 columns:
//   stream: a CU brings a phase's buffer at 60 KB/us for every block it gets;
//           0.25 us per phase and 4 us around them for every round of the
//           blocks that its LDS holds at once
//   tiles:  1.75 us per step of 128 columns, a block per CU at a time
// (2048 rows x 7168, 65 bf16 tokens: stream 15 us, tiles 99; 7168 x 7168, 300 of them:
// 101 and 100; 16384 x 2048, 300: 76 and 35. MXFP8 tokens: 15 and 109; 103 and 109; 86
// and 38.)
constexpr double kCus = 256.0;

template <int NM, bool X8, int NT>
double stream_us(const DenseParams &p)
{
    const double blocks = ceil(p.N / 32.0) * ceil(p.T / (16.0 * NT)), phases = ceil(ceil(p.K / 128.0) / kStC);
    constexpr int held = kMaxLds / st_lds<NM, X8, NT>() < 2 ? 1 : 2;   // blocks in a CU's LDS
    return ceil(blocks / kCus) * phases * (st_buf<NM, X8, NT>() / 1024 / 60.0) +
           ceil(blocks / (kCus * held)) * (phases * 0.25 + 4.0);
}

template <int NM, bool X8>
double tile_us(const DenseParams &p)
{
    const double blocks = ceil(p.N * (double)NM / kTlRows) * ceil(p.T / (double)kTlTok);
    return ceil(blocks / kCus) * ceil(p.K / 128.0) * 1.75 + 2.5;
}

// f(std::integral_constant<int, I>) for I in [B, E), on the host.
template <int B, int E, class F>
void each(F &&f)
{
    if constexpr (B < E) {
        f(std::integral_constant<int, B>{});
        each<B + 1, E>(f);
    }
}

// More than kGvTok tokens, or fewer whose rows the LDS of k_mx_gemv does not hold.
template <int NM, bool X8>
k3moe_status launch_batch(const DenseParams &p, hipStream_t s)
{
    // token tiles per block: as many as the LDS holds at most
    constexpr int most = X8 ? 4 : 5 - NM;
    double us = stream_us<NM, X8, 1>(p);
    int nt = 1;
    each<2, most + 1>([&](auto k) {
        constexpr int NT = decltype(k)::value;
        const double u = stream_us<NM, X8, NT>(p);
        if (u < us) us = u, nt = NT;
    });
    if (p.K >= 128 && tile_us<NM, X8>(p) < us) {
        const int64_t rb = ((int64_t)p.N * NM + kTlRows - 1) / kTlRows, tb = ((int64_t)p.T + kTlTok - 1) / kTlTok;
        if (rb * tb > kMaxItems / (64 * kTlWaves)) return K3MOE_E_UNSUPPORTED_SHAPE;
        launch_tile<NM, X8>(p, rb * tb, (int)tb, s);
        return K3MOE_OK;
    }
    k3moe_status st = K3MOE_E_UNSUPPORTED_SHAPE;
    each<1, most + 1>([&](auto k) {
        if (nt == decltype(k)::value) st = launch_stream<NM, X8, decltype(k)::value>(p, s);
    });
    return st;
}

template <int NM, bool X8>
void launch_few(const DenseParams &p, hipStream_t s)
{
    const int t1 = (int)(((int64_t)p.N + 15) / 16), t2 = (t1 + 1) / 2;
    if (p.kind == K3MOE_OUT_MXFP8) launch_gemv<NM, X8, true, 2>(p, 2 * t2, t1 < gv_long<NM, true>() ? t2 : kGvBlocks, s);
    else if (t1 < gv_long<NM, false>()) launch_gemv<NM, X8, false, 2>(p, t1, t1, s);
    else launch_gemv<NM, X8, false, 4>(p, t1, kGvBlocks, s);
}

template <int NM>
k3moe_status launch_dense(const DenseParams &p, hipStream_t s)
{
    k3moe_status st = K3MOE_OK;
    if (p.T <= kGvTok && (int64_t)p.T * 2 * p.K <= kGvMaxLds) {
        if (p.xs) launch_few<NM, true>(p, s);
        else launch_few<NM, false>(p, s);
    } else if (p.xs) {
        st = launch_batch<NM, true>(p, s);
    } else {
        st = launch_batch<NM, false>(p, s);
    }
    if (st != K3MOE_OK) return st;
    return hipGetLastError() == hipSuccess ? K3MOE_OK : K3MOE_E_HIP;
}

bool at(const void *q, size_t a) { return ((uintptr_t)q % a) == 0; }

// The checks that linear and glu share; fills the parameters. *nothing: no token.
k3moe_status check_dense(DenseParams &p, const uint8_t *const *w, const uint8_t *const *ws, int nm, int32_t rows,
                         int32_t cols, const void *x, int64_t x_stride, const uint8_t *xs, int64_t xs_stride,
                         int32_t T, void *out, int64_t out_stride, uint8_t *outs, int64_t outs_stride, int32_t kind,
                         bool *nothing)
{
    *nothing = false;
    if (T < 0 || rows <= 0 || cols <= 0) return K3MOE_E_INVALID_ARG;
    if (kind < K3MOE_OUT_BF16 || kind > K3MOE_OUT_MXFP8) return K3MOE_E_INVALID_ARG;
    if (cols % 32 || cols > kMaxCols) return K3MOE_E_UNSUPPORTED_SHAPE;
    if (T == 0) {
        *nothing = true;
        return K3MOE_OK;
    }
    const int64_t KB = cols / 32, G = ((int64_t)rows + 31) / 32;
    if (!x || !out || (kind == K3MOE_OUT_MXFP8) != (outs != nullptr)) return K3MOE_E_INVALID_ARG;
    for (int m = 0; m < nm; ++m)
        if (!w[m] || !ws[m]) return K3MOE_E_INVALID_ARG;
    if (T == 1) x_stride = cols, xs_stride = KB, out_stride = rows, outs_stride = G;  // one row: no stride is used
    if (x_stride < cols || (xs && xs_stride < KB) || out_stride < rows || (outs && outs_stride < G))
        return K3MOE_E_INVALID_ARG;
    if (T > 1 && x_stride > kMaxTokenStride) return K3MOE_E_UNSUPPORTED_SHAPE;
    for (int m = 0; m < nm; ++m)
        if (!at(w[m], 16) || !at(ws[m], 16)) return K3MOE_E_ALIGNMENT;
    if (!at(x, 16) || x_stride % (xs ? 16 : 8)) return K3MOE_E_ALIGNMENT;
    const size_t oe = kind == K3MOE_OUT_MXFP8 ? 1 : kind == K3MOE_OUT_BF16 ? 2 : 4;
    if (!at(out, oe)) return K3MOE_E_ALIGNMENT;
    p.vec = at(out, 4 * oe) && out_stride % 4 == 0;
    for (int m = 0; m < nm; ++m) p.w[m] = w[m], p.ws[m] = ws[m];
    p.x = x, p.xs = xs, p.out = out, p.outs = outs;
    p.xst = x_stride, p.xsst = xs_stride, p.ost = out_stride, p.osst = outs_stride;
    p.N = rows, p.K = cols, p.T = T, p.kind = kind;
    return K3MOE_OK;
}

}  // namespace
}  // namespace k3moe

using namespace k3moe;

extern "C" {

k3moe_status k3moe_linear(const uint8_t *packed, const uint8_t *scales, int32_t rows, int32_t cols, const void *x,
                          int64_t x_stride, const uint8_t *xs, int64_t xs_stride, int32_t T, void *out,
                          int64_t out_stride, uint8_t *outs, int64_t outs_stride, int32_t out_kind, void *stream)
{
    DenseParams p{};
    bool nothing;
    const k3moe_status st = check_dense(p, &packed, &scales, 1, rows, cols, x, x_stride, xs, xs_stride, T, out,
                                        out_stride, outs, outs_stride, out_kind, &nothing);
    if (st != K3MOE_OK || nothing) return st;
    return launch_dense<1>(p, static_cast<hipStream_t>(stream));
}

k3moe_status k3moe_glu(const uint8_t *gate_packed, const uint8_t *gate_scales, const uint8_t *up_packed,
                       const uint8_t *up_scales, int32_t rows, int32_t cols, const void *x, int64_t x_stride,
                       const uint8_t *xs, int64_t xs_stride, int32_t T, int32_t act, float situ_b1, float situ_b2,
                       void *out, int64_t out_stride, uint8_t *outs, int64_t outs_stride, int32_t out_kind,
                       void *stream)
{
    if (act != K3MOE_ACT_SITU && act != K3MOE_ACT_SWIGLU) return K3MOE_E_INVALID_ARG;
    if (act == K3MOE_ACT_SITU && !(situ_b1 > 0.0f && situ_b1 < INFINITY && situ_b2 > 0.0f && situ_b2 < INFINITY))
        return K3MOE_E_INVALID_ARG;
    if (out_kind == K3MOE_OUT_F32_ADD) return K3MOE_E_INVALID_ARG;
    const uint8_t *w[2] = {gate_packed, up_packed}, *ws[2] = {gate_scales, up_scales};
    DenseParams p{};
    p.act = act, p.b1 = situ_b1, p.b2 = situ_b2;
    bool nothing;
    const k3moe_status st = check_dense(p, w, ws, 2, rows, cols, x, x_stride, xs, xs_stride, T, out, out_stride,
                                        outs, outs_stride, out_kind, &nothing);
    if (st != K3MOE_OK || nothing) return st;
    return launch_dense<2>(p, static_cast<hipStream_t>(stream));
}

}  // extern "C"
