// The residual addition with the RMS norm behind it (k3moe_add_norm): per row
//   h' = fp32(h + d)                                (d bf16, fp32 or absent)
//   v  = fp32(fp32(h' * inv) * gamma),  inv = fp32(1 / sqrt(sum h'^2 / H + eps))
//   x  = bf16_RNE(v),  (q, qs) = MXFP8(v)            (either or both)
// with the sum of squares in fp64: the numbers of k3moe_step's norm (the
// "kimi-k3-in-c" README, §5 k3_rmsnorm), for a stream that still lacks the
// attention output.
//
// Bound by memory: h is read and written once, d read once, the tokens
// written once. A row of up to eight loads per thread (8192 columns, or 2048 where
// only single columns can be loaded) stays in its block's registers between
// the sum and the scaling; a wider one is read again, from the L2. Measured
// with d in bf16: 8192 tokens x 7168 to bf16 131 us (5.4 TB/s), to MXFP8 132; one
// token 4.4 us, a launch with one load, one reduction and one store; 32 tokens to
// MXFP8 5.7, a us of it the conversion of 28 values per thread; 8192 x 7167, an odd width, 163 us read again (229 with 32 loads held).
#include "k3moe_internal.h"
#include "k3moe_mx8.h"

namespace k3moe {
namespace {

struct AddNormParams {
    float *h;
    const void *d;
    const float *gamma;
    uint16_t *x;
    uint8_t *q, *qs;
    int64_t hs, ds, xs, qst, qss;  // row strides, elements
    int T, H;
    float eps;
};

constexpr int kNoD = 0, kDBf16 = 1, kDF32 = 2;
constexpr int kAnThreads = 256;
constexpr int kAnMaxWidth = 1 << 30;  // columns and a block's steps past them are counted in 32 bits

template <int VEC> struct Vals { float v[VEC]; };

template <int VEC>
__device__ __forceinline__ Vals<VEC> ld_f32(const float *p)
{
    Vals<VEC> r;
    if constexpr (VEC == 4) {
        const float4 a = *reinterpret_cast<const float4 *>(p);
        r.v[0] = a.x, r.v[1] = a.y, r.v[2] = a.z, r.v[3] = a.w;
    } else {
        r.v[0] = *p;
    }
    return r;
}

template <int VEC>
__device__ __forceinline__ void st_f32(float *p, const Vals<VEC> &a)
{
    if constexpr (VEC == 4) *reinterpret_cast<float4 *>(p) = float4{a.v[0], a.v[1], a.v[2], a.v[3]};
    else *p = a.v[0];
}

template <int VEC, int DK>
__device__ __forceinline__ Vals<VEC> ld_d(const void *d, int64_t o)
{
    if constexpr (DK == kDF32) {
        return ld_f32<VEC>(static_cast<const float *>(d) + o);
    } else {
        Vals<VEC> r;
        const uint16_t *p = static_cast<const uint16_t *>(d) + o;
        if constexpr (VEC == 4) {
            const uint2 a = *reinterpret_cast<const uint2 *>(p);
            r.v[0] = bf16f(a.x & 0xffffu), r.v[1] = bf16f(a.x >> 16);
            r.v[2] = bf16f(a.y & 0xffffu), r.v[3] = bf16f(a.y >> 16);
        } else {
            r.v[0] = bf16f(*p);
        }
        return r;
    }
}

// fp32 -> bf16, round to nearest even; NaN stays NaN.
__device__ __forceinline__ uint32_t an_bf16(float f) { return f != f ? 0x7fc0u : bf16_rne_u32(f); }

// The scaled values of VEC elements at column e (valid: inside the row).
template <int VEC>
__device__ __forceinline__ void an_store(const AddNormParams &p, int64_t t, int e, bool valid, const Vals<VEC> &y)
{
    if (p.x && valid) {
        uint16_t *xo = p.x + t * p.xs + e;
        if constexpr (VEC == 4)
            *reinterpret_cast<uint2 *>(xo) = uint2{an_bf16(y.v[0]) | (an_bf16(y.v[1]) << 16),
                                                   an_bf16(y.v[2]) | (an_bf16(y.v[3]) << 16)};
        else
            *xo = (uint16_t)an_bf16(y.v[0]);
    }
    if (p.q) {  // every lane takes part in the group's maximum
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < VEC; ++i) m = fmaxf(m, valid ? mx8_mag(y.v[i]) : 0.0f);
        m = VEC == 4 ? octet_max(m) : half_wave_max(m);
        const int s = mx8_exp(m);
        const float inv = mx8_inv(s);
        if (valid) {
            uint8_t *qo = p.q + t * p.qst + e;
            if constexpr (VEC == 4) {
                uint32_t w = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) w |= mx8_code(y.v[i], inv) << (8 * i);
                *reinterpret_cast<uint32_t *>(qo) = w;
            } else {
                *qo = (uint8_t)mx8_code(y.v[0], inv);
            }
            if (e % 32 == 0) p.qs[t * p.qss + e / 32] = (uint8_t)(s + 127);
        }
    }
}

// One block per row (rows beyond the grid in turn). Thread i holds columns
// VEC * (i + kAnThreads * j), j < NJ: a group of 32 columns lies in 32 / VEC
// neighbouring lanes. NJ == 0: a row of any width, in steps of 8 loads, read
// again for the scaling (a thread reads what it wrote itself). Columns past the
// row's end are read at its last ones, which another thread may be writing, and
// not used.
template <int VEC, int DK, int NJ>
__global__ __launch_bounds__(kAnThreads) void k_add_norm(AddNormParams p)
{
    __shared__ double red[kAnThreads / 64];
    const int tid = threadIdx.x;
    constexpr int B = NJ ? NJ : 8;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        float *h = p.h + t * p.hs;
        Vals<VEC> v[B], gm[B];
        double ss = 0.0;
        const int step = VEC * kAnThreads * B;
        for (int e0 = VEC * tid; e0 < (NJ ? VEC * tid + 1 : p.H); e0 += step) {
            Vals<VEC> dv[B];
#pragma unroll
            for (int j = 0; j < B; ++j) {
                const int e = min(e0 + VEC * kAnThreads * j, p.H - VEC);
                v[j] = ld_f32<VEC>(h + e);
                if constexpr (DK != kNoD) dv[j] = ld_d<VEC, DK>(p.d, t * p.ds + e);
                if constexpr (NJ != 0) gm[j] = ld_f32<VEC>(p.gamma + e);
            }
#pragma unroll
            for (int j = 0; j < B; ++j) {
                const int e = e0 + VEC * kAnThreads * j;
                const bool in = e < p.H;
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    if constexpr (DK != kNoD) v[j].v[i] += dv[j].v[i];
                    if (in) ss = fma((double)v[j].v[i], (double)v[j].v[i], ss);
                }
                if constexpr (DK != kNoD)
                    if (in) st_f32<VEC>(h + e, v[j]);
            }
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) ss += __shfl_xor(ss, o);
        if ((tid & 63) == 0) red[tid >> 6] = ss;
        __syncthreads();
        double tot = 0.0;
#pragma unroll
        for (int w = 0; w < kAnThreads / 64; ++w) tot += red[w];
        const float inv = (float)(1.0 / sqrt(tot / (double)p.H + (double)p.eps));
        // every lane of the block makes the same number of steps (the groups' maxima need them all)
        for (int c0 = 0; c0 < (NJ ? 1 : p.H); c0 += step) {
            const int e0 = c0 + VEC * tid;
            if constexpr (NJ == 0) {
#pragma unroll
                for (int j = 0; j < B; ++j) {
                    const int e = e0 + VEC * kAnThreads * j;
                    const int ec = min(e, p.H - VEC);
                    if (e < p.H) v[j] = ld_f32<VEC>(h + e);  // a column of its own: what this thread wrote
                    gm[j] = ld_f32<VEC>(p.gamma + ec);
                }
            }
#pragma unroll
            for (int j = 0; j < B; ++j) {
                const int e = e0 + VEC * kAnThreads * j;
                Vals<VEC> y;
#pragma unroll
                for (int i = 0; i < VEC; ++i) y.v[i] = v[j].v[i] * inv * gm[j].v[i];
                an_store<VEC>(p, t, e, e < p.H, y);
            }
        }
        __syncthreads();  // red is free for the next row
    }
}

template <int VEC, int DK>
void launch_add_norm(const AddNormParams &p, hipStream_t s)
{
    const unsigned grid = (unsigned)(p.T < (1 << 20) ? p.T : (1 << 20));
    const int per = (p.H + VEC * kAnThreads - 1) / (VEC * kAnThreads);  // loads per thread
    // 8192 rows of bf16: 2048 wide 38 us with two loads per thread, 68 with eight; 4096 wide 73 with four, 84 with eight
    if (per > 8) {
        k_add_norm<VEC, DK, 0><<<grid, kAnThreads, 0, s>>>(p);
    } else if constexpr (VEC == 4) {
        if (per <= 2) k_add_norm<VEC, DK, 2><<<grid, kAnThreads, 0, s>>>(p);
        else if (per <= 4) k_add_norm<VEC, DK, 4><<<grid, kAnThreads, 0, s>>>(p);
        else k_add_norm<VEC, DK, 8><<<grid, kAnThreads, 0, s>>>(p);
    } else {
        k_add_norm<VEC, DK, 8><<<grid, kAnThreads, 0, s>>>(p);
    }
}

bool at(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

}  // namespace
}  // namespace k3moe

using namespace k3moe;

extern "C" k3moe_status k3moe_add_norm(float *h, int64_t h_stride, const void *d, int32_t d_kind, int64_t d_stride,
                                       int32_t T, int32_t H, const float *gamma, float eps, uint16_t *x,
                                       int64_t x_stride, uint8_t *q, int64_t q_stride, uint8_t *qs,
                                       int64_t qs_stride, void *stream)
{
    if (T < 0 || H <= 0 || !(eps > 0.0f && eps < INFINITY)) return K3MOE_E_INVALID_ARG;
    if (H > kAnMaxWidth) return K3MOE_E_UNSUPPORTED_SHAPE;
    if (d ? d_kind != K3MOE_ADD_BF16 && d_kind != K3MOE_ADD_F32 : d_kind != K3MOE_ADD_NONE)
        return K3MOE_E_INVALID_ARG;
    if (T == 0) return K3MOE_OK;
    if (!h || !gamma || (!x && !q) || (q == nullptr) != (qs == nullptr)) return K3MOE_E_INVALID_ARG;
    const int64_t G = ((int64_t)H + 31) / 32;
    if (T == 1) h_stride = d_stride = x_stride = q_stride = H, qs_stride = G;  // one row: no stride is used
    if (h_stride < H || (d && d_stride < H) || (x && x_stride < H) || (q && (q_stride < H || qs_stride < G)))
        return K3MOE_E_INVALID_ARG;
    const size_t de = d_kind == K3MOE_ADD_BF16 ? 2 : 4;
    if (!at(h, 4) || !at(gamma, 4) || (d && !at(d, de)) || (x && !at(x, 2))) return K3MOE_E_ALIGNMENT;
    AddNormParams p{};
    p.h = h, p.d = d, p.gamma = gamma, p.x = x, p.q = q, p.qs = qs;
    p.hs = h_stride, p.ds = d_stride, p.xs = x_stride, p.qst = q_stride, p.qss = qs_stride;
    p.T = T, p.H = H, p.eps = eps;
    // four columns per load where the width, the bases and the strides of every tensor allow it
    const bool v4 = H % 4 == 0 && at(h, 16) && at(gamma, 16) && (T == 1 || h_stride % 4 == 0) &&
                    (!d || (at(d, 4 * de) && d_stride % 4 == 0)) && (!x || (at(x, 8) && x_stride % 4 == 0)) &&
                    (!q || (at(q, 4) && q_stride % 4 == 0));
    hipStream_t s = static_cast<hipStream_t>(stream);
    switch (d ? d_kind : 0) {
    case K3MOE_ADD_BF16:
        v4 ? launch_add_norm<4, kDBf16>(p, s) : launch_add_norm<1, kDBf16>(p, s);
        break;
    case K3MOE_ADD_F32:
        v4 ? launch_add_norm<4, kDF32>(p, s) : launch_add_norm<1, kDF32>(p, s);
        break;
    default:
        v4 ? launch_add_norm<4, kNoD>(p, s) : launch_add_norm<1, kNoD>(p, s);
    }
    return hipGetLastError() == hipSuccess ? K3MOE_OK : K3MOE_E_HIP;
}
