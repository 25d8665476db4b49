// Dense products with MXFP4 matrices (k3moe_linear) and the gated pair of them
// (k3moe_glu):
//   y[t][n] = sum_k W[n][k] x[t][k],   a[t][n] = act(W1 x, W3 x)
// on bf16 or MXFP8 tokens. The format is the one of the experts (the
// "kimi-k3-in-c" README, §4 "Reduction one: the experts already ship at half a
// byte"), the activation §9's k3_situ_glu.
//
// Weights and 8-bit tokens are expanded to bf16 in registers, which is exact
// (an fp4 or e4m3 value times a power of two is a bf16), and multiplied on
// v_mfma_f32_16x16x32_bf16: exact products, fp32 sums.
//
// K mapping. A lane's 16-byte weight load holds one 32-weight block of its
// row: lane 16g + r of an MFMA tile loads block 4c + g of row r in chunk c (128
// columns), and step s of the chunk multiplies columns 128c + 32g + 8s + [0, 8)
// of every g; the token side reads the same columns.
#include "k3moe_internal.h"
#include "k3moe_mx8.h"

namespace k3moe {
namespace {

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
};

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

// A block owns 32 rows of each matrix and 16 tokens; its waves take the chunks
// of 128 columns in turn, and their fp32 sums are added in wave order.
constexpr int kStW = 4;

template <int NM, bool X8>
__global__ __launch_bounds__(64 * kStW) void k_mx_stream(DenseParams p, int row_blocks)
{
    __shared__ float4 red[kStW][NM][2][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, l16 = lane & 15;
    const int rb = blockIdx.x % row_blocks, tb = blockIdx.x / row_blocks;
    const int n0 = 32 * rb, t0 = 16 * tb;
    const int KB = p.K / 32, NC = (KB + 3) / 4;
    const int64_t tx = min(t0 + l16, p.T - 1);
    const uint8_t *wr[NM][2], *sr[NM][2];
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int64_t n = min(n0 + 16 * r + l16, p.N - 1);
            wr[m][r] = p.w[m] + n * (p.K / 2);
            sr[m][r] = p.ws[m] + n * KB;
        }
    v4f acc[NM][2];
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r) acc[m][r] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    for (int c = wave; c < NC; c += kStW) {
        const int kb = 4 * c + g;
        const bool ok = kb < KB;   // past the last block: zeros on both sides
        const int kc = ok ? kb : KB - 1;
        bf8 b[4];
        if constexpr (X8) {
            const u4 *xp = reinterpret_cast<const u4 *>(static_cast<const uint8_t *>(p.x) + tx * p.xst + 32 * kc);
            u4 x0 = xp[0], x1 = xp[1];
            const uint32_t sx = p.xs[tx * p.xsst + kc];
            if (!ok || sx == 255u) x0 = x1 = u4{0u, 0u, 0u, 0u};
            const float f = e8m0_to_f32(sx);
            b[0] = expand8_fp8(x0.x, x0.y, f), b[1] = expand8_fp8(x0.z, x0.w, f);
            b[2] = expand8_fp8(x1.x, x1.y, f), b[3] = expand8_fp8(x1.z, x1.w, f);
        } else {
            const u4 *xp = reinterpret_cast<const u4 *>(static_cast<const uint16_t *>(p.x) + tx * p.xst + 32 * kc);
#pragma unroll
            for (int s = 0; s < 4; ++s) b[s] = as_bf8(ok ? xp[s] : u4{0u, 0u, 0u, 0u});
        }
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                u4 a = *reinterpret_cast<const u4 *>(wr[m][r] + 16 * kc);
                const uint32_t sw = sr[m][r][kc];
                if (!ok || sw == 255u) a = u4{0u, 0u, 0u, 0u};
                const float f = e8m0_to_f32(sw);
#pragma unroll
                for (int s = 0; s < 4; ++s) acc[m][r] = mfma_bf16(dequant8_bf16(a[s], f), b[s], acc[m][r]);
            }
    }
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r)  // [token][row]: lane l16 holds rows 4g + i of token l16
            red[wave][m][r][4 * l16 + g] = float4{acc[m][r][0], acc[m][r][1], acc[m][r][2], acc[m][r][3]};
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int tok = (tid >> 5) + 8 * q, row = tid & 31;
        float v[NM];
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            v[m] = 0.0f;
#pragma unroll
            for (int w = 0; w < kStW; ++w)
                v[m] += reinterpret_cast<const float *>(&red[w][m][row >> 4][0])[16 * tok + (row & 15)];
        }
        float y = v[0];
        if constexpr (NM == 2) y = act_fn(v[0], v[1], p.act, p.b1, p.b2);
        dense_store(p, t0 + tok, n0 + row, t0 + tok < p.T && n0 + row < p.N, y);
    }
}

// work-items of a launch are counted in 32 bits
constexpr int64_t kMaxItems = ((int64_t)1 << 32) - 1;

template <int NM>
k3moe_status launch_dense(const DenseParams &p, hipStream_t s)
{
    const int64_t rb = ((int64_t)p.N + 31) / 32, tb = ((int64_t)p.T + 15) / 16;
    if (rb * tb > kMaxItems / (64 * kStW)) return K3MOE_E_UNSUPPORTED_SHAPE;
    if (p.xs) k_mx_stream<NM, true><<<(unsigned)(rb * tb), 64 * kStW, 0, s>>>(p, (int)rb);
    else k_mx_stream<NM, false><<<(unsigned)(rb * tb), 64 * kStW, 0, s>>>(p, (int)rb);
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
    if (cols % 32) return K3MOE_E_UNSUPPORTED_SHAPE;
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
    for (int m = 0; m < nm; ++m)
        if (!at(w[m], 16) || !at(ws[m], 16)) return K3MOE_E_ALIGNMENT;
    if (!at(x, 16) || x_stride % (xs ? 16 : 8)) return K3MOE_E_ALIGNMENT;
    if (!at(out, kind == K3MOE_OUT_MXFP8 ? 1 : kind == K3MOE_OUT_BF16 ? 2 : 4)) return K3MOE_E_ALIGNMENT;
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
