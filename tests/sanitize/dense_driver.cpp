// Drives the host-side checks of the dense operators (argument refusals, empty
// batches, grids past 32 bits with their time models) for a build of their host
// code with AddressSanitizer and UndefinedBehaviorSanitizer. Every call here
// returns before the first HIP runtime call, so it runs without a GPU. Prints
// "ok" and exits 0 when each status is the one the header documents.
#include <cmath>
#include <cstdint>
#include <cstdio>

#include "k3moe.h"

// The HIP runtime keeps process-lifetime allocations of its own.
extern "C" const char *__asan_default_options() { return "detect_leaks=0"; }

static int failures = 0;

#define EXPECT(call, want)                                                                    \
    do {                                                                                      \
        const int got_ = (int)(call);                                                         \
        if (got_ != (int)(want)) {                                                            \
            std::fprintf(stderr, "%s:%d: %s gave %d, want %d\n", __FILE__, __LINE__, #call, got_, \
                         (int)(want));                                                        \
            failures++;                                                                       \
        }                                                                                     \
    } while (0)

// An address that is only tested for presence and alignment.
static uint8_t *at(uintptr_t off = 0) { return reinterpret_cast<uint8_t *>((uintptr_t)0x10000000 + off); }

static k3moe_status norm(int32_t T, int32_t H, int64_t st, float eps, uint8_t *h)
{
    return k3moe_add_norm(reinterpret_cast<float *>(h), st, at(), K3MOE_ADD_BF16, st, T, H,
                          reinterpret_cast<const float *>(at()), eps, reinterpret_cast<uint16_t *>(at()), st, nullptr,
                          0, nullptr, 0, nullptr);
}

static k3moe_status linear(int32_t N, int32_t K, int32_t T, int64_t xst, int64_t ost, uint8_t *xs, uint8_t *x, int kind)
{
    return k3moe_linear(at(), at(), N, K, x, xst, xs, xst / 32, T, at(), ost, kind == K3MOE_OUT_MXFP8 ? at() : nullptr,
                        ost / 32 + 1, kind, nullptr);
}

int main()
{
    const int32_t big = INT32_MAX;
    EXPECT(norm(0, 64, 64, 1e-5f, nullptr), K3MOE_OK);
    EXPECT(norm(-1, 64, 64, 1e-5f, at()), K3MOE_E_INVALID_ARG);
    EXPECT(norm(2, 0, 64, 1e-5f, at()), K3MOE_E_INVALID_ARG);
    EXPECT(norm(2, big, big, 1e-5f, at()), K3MOE_E_UNSUPPORTED_SHAPE);
    EXPECT(norm(2, 64, INT64_MIN, 1e-5f, at()), K3MOE_E_INVALID_ARG);
    EXPECT(norm(2, 64, 64, -1e-5f, at()), K3MOE_E_INVALID_ARG);
    EXPECT(norm(2, 64, 64, INFINITY, at()), K3MOE_E_INVALID_ARG);
    EXPECT(norm(2, 64, 64, 1e-5f, nullptr), K3MOE_E_INVALID_ARG);
    EXPECT(norm(2, 64, 64, 1e-5f, at(2)), K3MOE_E_ALIGNMENT);
    for (int kind = 1; kind <= 4; ++kind)
        for (int f8 = 0; f8 < 2; ++f8) {
            uint8_t *xs = f8 ? at() : nullptr;
            EXPECT(linear(64, 64, 0, 64, 64, xs, nullptr, kind), K3MOE_OK);
            EXPECT(linear(64, 64, -1, 64, 64, xs, at(), kind), K3MOE_E_INVALID_ARG);
            EXPECT(linear(64, 65, 2, 128, 64, xs, at(), kind), K3MOE_E_UNSUPPORTED_SHAPE);
            EXPECT(linear(64, big - 31, 2, big, 64, xs, at(), kind), K3MOE_E_UNSUPPORTED_SHAPE);
            EXPECT(linear(64, 64, 2, INT64_MIN, 64, xs, at(), kind), K3MOE_E_INVALID_ARG);
            EXPECT(linear(64, 64, 2, 64, 63, xs, at(), kind), K3MOE_E_INVALID_ARG);
            EXPECT(linear(64, 64, 2, 64, 64, xs, at(8), kind), K3MOE_E_ALIGNMENT);
            // grids past 32 bits: through the time models of every token kind
            EXPECT(linear(big, 32, big, 32, (int64_t)big + 1, xs, at(), kind), K3MOE_E_UNSUPPORTED_SHAPE);
            EXPECT(linear(big, 4096, big, 4096, (int64_t)big + 1, xs, at(), kind), K3MOE_E_UNSUPPORTED_SHAPE);
            EXPECT(linear(32, 4096, big, (int64_t)1 << 40, 64, xs, at(), kind), K3MOE_E_UNSUPPORTED_SHAPE);
        }
    EXPECT(k3moe_glu(at(), at(), at(), at(), big, 4096, at(), 4096, nullptr, 0, big, K3MOE_ACT_SITU, 4.0f, 25.0f, at(),
                     (int64_t)big + 1, nullptr, 0, K3MOE_OUT_BF16, nullptr),
           K3MOE_E_UNSUPPORTED_SHAPE);
    EXPECT(k3moe_glu(at(), at(), at(), at(), 64, 64, at(), 64, nullptr, 0, 2, K3MOE_ACT_SITU, NAN, 25.0f, at(), 64,
                     nullptr, 0, K3MOE_OUT_BF16, nullptr),
           K3MOE_E_INVALID_ARG);
    EXPECT(k3moe_glu(at(), at(), at(), at(), 64, 64, at(), 64, nullptr, 0, 2, 7, 4.0f, 25.0f, at(), 64, nullptr, 0,
                     K3MOE_OUT_BF16, nullptr),
           K3MOE_E_INVALID_ARG);
    if (failures) return 1;
    std::puts("ok");
    return 0;
}
