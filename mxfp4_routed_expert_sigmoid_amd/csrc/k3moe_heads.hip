// Norm of query and key heads, rotation by position, and the write of keys and
// values into the cache (k3moe_qk_norm_rope). Per head x of width D:
//   n  = x * inv * gamma,  inv = 1 / sqrt(sum x^2 / D + eps)
//   a  = position * inv_freq[i]
//   y1 = n1 cos a - n2 sin a,  y2 = n2 cos a + n1 sin a
// with (1, 2) = (i, i + R / 2) or (2 i, 2 i + 1) for the first R dimensions.
//
// A lane holds 8 neighbouring dimensions (16 bytes) of a head, so one wave
// instruction moves 64 / lanes heads, whole lines of them; the heads of a
// token that a wave handles have the same angles, which it takes once: in 64
// bits up to the fraction of a turn (an fp32 product of a position of 10^6 would
// be off by 0.06 of a radian), the sine and cosine of that fraction in 32.
//
// Bound by memory: 8192 tokens of 64 + 8 heads of 128 with keys and values into
// a bf16 cache 73 to 78 us (352 MB, 4.5 to 4.8 TB/s, a large copy's rate).
// Eight heads a lane are in flight, their loads in front of the angles' 64-bit
// products; the sum over a head's lanes and the exchange of halves go through
// DPP, not the LDS. One token: 5.5 us in a graph, the launch and two latencies.
#include "k3moe_internal.h"
#include "k3moe_mx8.h"

namespace k3moe {
namespace {

constexpr int kHdThreads = 256, kHdBatch = 8;   // heads in flight per lane
constexpr int kHdMaxTokens = 1 << 25;           // a launch's work-items are counted in 32 bits

struct HeadsParams {
    const uint16_t *q, *k, *v;
    uint16_t *qo, *ko;
    const float *gq, *gk, *freq;
    const int32_t *pos;
    const int64_t *slots;
    uint8_t *kc, *vc, *ks, *vs;
    int64_t qs, kst, vst, qos, kos, places;
    int T, Hq, Hkv, D, Dv, R, rot, page, lpage, split;
    int qi, ki, vi;   // steps of a token: queries, keys, values
    float eps, per_dim;   // 1 / D
};

// Eight fp32 -> bf16, to nearest even; NaN stays NaN.
__device__ __forceinline__ u4 hd_pack(const float (&y)[8])
{
    typedef float f8 __attribute__((ext_vector_type(8)));
    const bf8 b = __builtin_convertvector((f8{y[0], y[1], y[2], y[3], y[4], y[5], y[6], y[7]}), bf8);
    u4 r;
    __builtin_memcpy(&r, &b, 16);
    return r;
}

__device__ __forceinline__ void hd_unpack(u4 w, float (&x)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = bf16f(w[i] & 0xffffu), x[2 * i + 1] = bf16f(w[i] >> 16);
}

template <int CTRL>
__device__ __forceinline__ float hd_dpp(float v)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, false));
}

// Sum over LH lanes, in each of them.
template <int LH>
__device__ __forceinline__ float hd_sum(float v)
{
    v += hd_dpp<0xb1>(v);                        // neighbours
    v += hd_dpp<0x4e>(v);                        // pairs
    v += hd_dpp<0x141>(v);                       // mirrored eights
    if constexpr (LH > 8) v += hd_dpp<0x140>(v); // mirrored sixteens
    if constexpr (LH > 16) v += __shfl_xor(v, 16);
    return v;
}

// The value of the lane LH / 2 away among LH.
template <int LH>
__device__ __forceinline__ float hd_half(float v)
{
    if constexpr (LH == 8) return hd_dpp<0x1b>(hd_dpp<0x141>(v));   // 7 - i, then i ^ 3
    if constexpr (LH == 16) return hd_dpp<0x128>(v);                // turned by eight
    return __shfl_xor(v, 16);
}

// Maximum over the four lanes of a quad.
__device__ __forceinline__ float quad_max(float m)
{
    m = fmaxf(m, hd_dpp<0xb1>(m));
    return fmaxf(m, hd_dpp<0x4e>(m));
}

// Eight values of row `row` of the cache at dimension e: bf16, or MXFP8 with the quad's lanes holding one group.
// Every lane of a quad takes part; in: the place exists.
__device__ __forceinline__ void hd_cache(uint8_t *c, uint8_t *s, int64_t row, int dim, int e, bool in, const float (&y)[8])
{
    if (!s) {
        if (in) *reinterpret_cast<u4 *>(c + 2 * (row * dim + e)) = hd_pack(y);
        return;
    }
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, in ? mx8_mag(y[i]) : 0.0f);
    const int x = mx8_exp(quad_max(m));
    if (!in) return;
    const float inv = mx8_inv(x);
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i >> 2] |= mx8_code(y[i], inv) << (8 * (i & 3));
    *reinterpret_cast<uint2 *>(c + row * dim + e) = uint2{w[0], w[1]};
    if (e % 32 == 0) s[row * (dim / 32) + e / 32] = (uint8_t)(x + 127);
}

// Sine and cosine of t turns, |t| <= 1/2: the angle from the nearest quarter turn, r in [-pi/4, pi/4], and the series of
// both there (their next terms, r^11 / 11! and r^10 / 10!, are below 2^-28 and 2^-25).
__device__ __forceinline__ void turn_sincos(float t, float &s, float &c)
{
    const float q = rintf(4.0f * t), r = fmaf(q, -0.25f, t) * 6.28318531f, z = r * r;
    const float a = fmaf(z * r, fmaf(z, fmaf(z, fmaf(z, 2.75573192e-6f, -1.98412698e-4f), 8.33333333e-3f), -0.166666667f), r);
    const float b = fmaf(z, fmaf(z, fmaf(z, fmaf(z, 2.48015873e-5f, -1.38888889e-3f), 4.16666667e-2f), -0.5f), 1.0f);
    const int k = (int)q;
    const float x = k & 1 ? b : a, y = k & 1 ? a : b;
    s = k & 2 ? -x : x;
    c = (k + 1) & 2 ? -y : y;
}

// LH lanes per head (D <= 8 LH). Wave w of token w / split takes the token's steps w % split, + split, ...: first the
// queries' (64 / LH heads each), then the keys', then the values' (64 pieces of 16 bytes each).
template <int LH>
__global__ __launch_bounds__(kHdThreads) void k_heads(HeadsParams p)
{
    constexpr int HW = 64 / LH;
    const int lane = threadIdx.x & 63, sub = lane % LH, e0 = 8 * sub;
    const int64_t w = (int64_t)blockIdx.x * (kHdThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = (int)(w / p.split), part = (int)(w % p.split);
    if (t >= p.T) return;
    const bool used = e0 < p.D;
    const int ec = used ? e0 : 0;
    const int64_t slot = p.slots ? p.slots[t] : -1;
    const bool place = slot >= 0 && slot < p.places;
    const int64_t prow = place ? (slot >> p.lpage) * p.Hkv * p.page + (slot & (p.page - 1)) : 0;   // row of head 0

    // Sine and cosine for this lane's eight dimensions (0 and 1 behind the rotated ones), taken behind the first loads.
    const bool turns = e0 < p.R, pairs = p.rot == K3MOE_ROT_PAIRS;
    const int pos = p.R > 0 ? p.pos[t] : 0;
    float freq[8], cs[8], sn[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int i = pairs ? (e0 + j) / 2 : e0 + j < p.R / 2 ? e0 + j : e0 + j - p.R / 2;
        freq[j] = turns ? p.freq[i] : 0.0f;
    }
    bool ready = false;
    auto angles = [&]() {
        if (ready) return;
        ready = true;
        const double at = (double)pos * 0.15915494309189535;   // 1 / (2 pi)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j & 1) {
                if (pairs) {
                    cs[j] = cs[j - 1], sn[j] = sn[j - 1];
                    continue;
                }
            }
            const double turn = at * (double)freq[j];
            turn_sincos((float)(turn - rint(turn)), sn[j], cs[j]);
        }
    };
    // y1 = n1 c - n2 s, y2 = n2 c + n1 s: the second of a pair takes its sine with the other sign
    const bool first = e0 < p.R / 2;
    const int other = turns ? (lane - sub) + (first ? sub + p.R / 16 : sub - p.R / 16) : lane;

    auto run = [&](const uint16_t *x, int H, int s0, int steps, const float *gamma, uint16_t *out, bool cached) {
        float g[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = gamma ? gamma[ec + j] : 1.0f;
        for (int s = s0; s < steps; s += kHdBatch * p.split) {
            u4 raw[kHdBatch];
#pragma unroll
            for (int b = 0; b < kHdBatch; ++b) {
                const int head = min((s + b * p.split) * HW + lane / LH, H - 1);
                raw[b] = *reinterpret_cast<const u4 *>(x + head * p.D + ec);
            }
            angles();
#pragma unroll
            for (int b = 0; b < kHdBatch; ++b) {
                if (s + b * p.split >= steps) break;     // the same for the whole wave
                const int head = (s + b * p.split) * HW + lane / LH;
                const bool in = used && head < H;
                float y[8];
                hd_unpack(raw[b], y);
                if (gamma) {
                    float ss = 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) ss = fmaf(y[j], y[j], ss);
                    const float mean = fmaf(hd_sum<LH>(used ? ss : 0.0f), p.per_dim, p.eps);
                    float inv = __builtin_amdgcn_rsqf(mean);   // within an ulp
                    // squares that fp32 does not hold (or digits of theirs): those heads once more, scaled
                    if (__ballot(!(mean >= 0x1p-100f && mean < INFINITY))) {
                        const float by = mean < INFINITY ? mean >= 0x1p-100f ? 1.0f : 0x1p70f : 0x1p-70f;
                        ss = 0.0f;
#pragma unroll
                        for (int j = 0; j < 8; ++j) ss = fmaf(y[j] * by, y[j] * by, ss);
                        inv = __builtin_amdgcn_rsqf(fmaf(hd_sum<LH>(used ? ss : 0.0f), p.per_dim, p.eps * by * by)) * by;
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] = y[j] * inv * g[j];
                }
                if (p.R > 0) {
                    float z[8];
                    if (pairs) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) z[j] = y[j ^ 1];
                    } else if (p.R == 8 * LH) {      // the whole head: the lane half a head away
#pragma unroll
                        for (int j = 0; j < 8; ++j) z[j] = hd_half<LH>(y[j]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) z[j] = __shfl(y[j], other);
                    }
                    if (turns) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            y[j] = fmaf(y[j], cs[j], (pairs ? (j & 1) == 0 : first) ? -(z[j] * sn[j]) : z[j] * sn[j]);
                    }
                }
                if (out && in) *reinterpret_cast<u4 *>(out + head * p.D + e0) = hd_pack(y);
                if (cached && place)
                    hd_cache(p.kc, p.ks, prow + (int64_t)head * p.page, p.D, e0, in, y);
            }
        }
    };
    if (p.qo) {
        run(p.q + t * p.qs, p.Hq, part, p.qi, p.gq, p.qo + t * p.qos, false);
    }
    // the keys' steps go on behind the queries': the waves' shares stay even
    const int k0 = (part + p.split - p.qi % p.split) % p.split;
    if (p.ko || p.kc) run(p.k + t * p.kst, p.Hkv, k0, p.ki, p.gk, p.ko ? p.ko + t * p.kos : nullptr, p.kc != nullptr);
    if (!place) return;
    const int v0 = (part + p.split - (p.qi + p.ki) % p.split) % p.split, pieces = p.Dv / 8;
    for (int s = v0; s < p.vi; s += p.split) {
        const int at = 64 * s + lane, head = at / pieces, e = 8 * (at - head * pieces);
        const bool in = head < p.Hkv;
        float y[8];
        hd_unpack(*reinterpret_cast<const u4 *>(p.v + t * p.vst + (in ? 8 * at : 0)), y);
        hd_cache(p.vc, p.vs, prow + (int64_t)head * p.page, p.Dv, e, in, y);
    }
}

template <int LH>
void launch_heads(HeadsParams p, hipStream_t s)
{
    constexpr int HW = 64 / LH;
    p.qi = p.qo ? (p.Hq + HW - 1) / HW : 0;
    p.ki = p.ko || p.kc ? (p.Hkv + HW - 1) / HW : 0;
    p.vi = p.kc ? (p.Hkv * p.Dv / 8 + 63) / 64 : 0;
    // One wave per token where that gives the card its 2048 waves; few tokens are split over more of them, up to a step
    // each. One wave and this, tokens of 64 + 8 heads of 128: 1: 10.9 and 5.2 us, 64: 11.9 and 7.2, 256: 12.2 and 8.8,
    // 1024: 15.1 and 14.0; 8192 waves: 15.7 at 256, 28 at 2048 (20.4 with one each), as every wave takes the angles anew.
    const int steps = max(p.qi + p.ki + p.vi, 1);
    p.split = min(steps, (2048 + p.T - 1) / p.T);
    const int64_t waves = (int64_t)p.T * p.split;
    k_heads<LH><<<(unsigned)((waves + 3) / 4), kHdThreads, 0, s>>>(p);
}

bool at(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

}  // namespace
}  // namespace k3moe

using namespace k3moe;

extern "C" k3moe_status k3moe_qk_norm_rope(const uint16_t *q, int64_t q_stride, const uint16_t *k, int64_t k_stride,
                                           const uint16_t *v, int64_t v_stride, int32_t T, int32_t q_heads,
                                           int32_t kv_heads, int32_t dim, int32_t v_dim, const float *gamma_q,
                                           const float *gamma_k, float eps, const int32_t *positions,
                                           const float *inv_freq, int32_t rot_dim, int32_t rot_kind, uint16_t *q_out,
                                           int64_t q_out_stride, uint16_t *k_out, int64_t k_out_stride,
                                           const k3moe_pages *cache, const int64_t *slots, void *stream)
{
    if (T < 0 || q_heads <= 0 || kv_heads <= 0 || dim <= 0 || rot_dim < 0 || rot_dim > dim || !(eps > 0.0f && eps < INFINITY) ||
        (rot_kind != K3MOE_ROT_HALVES && rot_kind != K3MOE_ROT_PAIRS) || (inv_freq == nullptr) != (rot_dim == 0) ||
        (cache && v_dim <= 0))
        return K3MOE_E_INVALID_ARG;
    const bool x8 = cache && cache->ks;
    if (T > kHdMaxTokens || dim % 8 || dim > 256 || q_heads > 4096 || kv_heads > 4096 || rot_dim % 16 || (cache && (v_dim % 8 || v_dim > 256)) ||
        (x8 && (dim % 32 || v_dim % 32)))
        return K3MOE_E_UNSUPPORTED_SHAPE;
    if (cache) {
        const int page = cache->page;
        if (cache->pages < 0 || page <= 0 || (cache->vs != nullptr) != x8) return K3MOE_E_INVALID_ARG;
        if (page < 16 || page > 1 << 20 || (page & (page - 1))) return K3MOE_E_UNSUPPORTED_SHAPE;
        if (cache->pages > 0 && (!cache->k || !cache->v)) return K3MOE_E_INVALID_ARG;
    }
    if (T == 0) return K3MOE_OK;
    if (!q || !k || (!q_out && !k_out && !cache) || (rot_dim > 0 && !positions) ||
        (cache == nullptr) != (slots == nullptr) || (cache == nullptr) != (v == nullptr))
        return K3MOE_E_INVALID_ARG;
    const int64_t qw = (int64_t)q_heads * dim, kw = (int64_t)kv_heads * dim, vw = (int64_t)kv_heads * v_dim;
    if (T == 1) q_stride = q_out_stride = qw, k_stride = k_out_stride = kw, v_stride = vw;
    if (q_stride < qw || k_stride < kw || (v && v_stride < vw) || (q_out && q_out_stride < qw) || (k_out && k_out_stride < kw))
        return K3MOE_E_INVALID_ARG;
    if (!at(q, 16) || !at(k, 16) || !at(v, 16) || !at(q_out, 16) || !at(k_out, 16) || q_stride % 8 || k_stride % 8 ||
        (v && v_stride % 8) || (q_out && q_out_stride % 8) || (k_out && k_out_stride % 8) || !at(gamma_q, 4) || !at(gamma_k, 4) ||
        !at(positions, 4) || !at(inv_freq, 4) || !at(slots, 8) || (cache && (!at(cache->k, 16) || !at(cache->v, 16))))
        return K3MOE_E_ALIGNMENT;
    HeadsParams p{};
    p.q = q, p.k = k, p.v = v, p.qo = q_out, p.ko = k_out, p.gq = gamma_q, p.gk = gamma_k, p.freq = inv_freq;
    p.pos = positions, p.slots = slots;
    p.qs = q_stride, p.kst = k_stride, p.vst = v_stride, p.qos = q_out_stride, p.kos = k_out_stride;
    p.T = T, p.Hq = q_heads, p.Hkv = kv_heads, p.D = dim, p.Dv = v_dim, p.R = rot_dim, p.rot = rot_kind, p.eps = eps, p.per_dim = 1.0f / (float)dim;
    if (cache && cache->pages > 0) {
        p.kc = static_cast<uint8_t *>(cache->k), p.vc = static_cast<uint8_t *>(cache->v), p.ks = cache->ks, p.vs = cache->vs;
        p.page = cache->page, p.lpage = __builtin_ctz((unsigned)cache->page), p.places = (int64_t)cache->pages * cache->page;
    }
    if (!p.qo && !p.ko && !p.kc) return K3MOE_OK;   // a cache without pages: nothing to write
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (dim <= 64) launch_heads<8>(p, s);
    else if (dim <= 128) launch_heads<16>(p, s);
    else launch_heads<32>(p, s);
    return hipGetLastError() == hipSuccess ? K3MOE_OK : K3MOE_E_HIP;
}
