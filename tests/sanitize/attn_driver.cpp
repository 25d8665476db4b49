// Drives the host-side checks of the attention operators (argument refusals,
// empty batches, workspace sizes, grids past 32 bits) for a build of their host
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
template <class T> static T *at(uintptr_t off = 0) { return reinterpret_cast<T *>((uintptr_t)0x10000000 + off); }
typedef uint16_t h16;

static k3moe_status heads(int32_t T, int32_t Hq, int32_t D, int64_t st, int32_t R, float eps, const k3moe_pages *c)
{
    return k3moe_qk_norm_rope(at<h16>(), st, at<h16>(), st, c ? at<h16>() : nullptr, st, T, Hq, 1, D, D, nullptr, nullptr,
                              eps, at<int32_t>(), R ? at<float>() : nullptr, R, K3MOE_ROT_HALVES, at<h16>(2), st, nullptr, 0, c,
                              c ? at<int64_t>() : nullptr, nullptr);
}

static k3moe_status att(int32_t seqs, int32_t T, int32_t Hq, int32_t Hkv, int64_t st, float scale, uintptr_t off)
{
    return k3moe_attention(at<h16>(off), st, at<h16>(), st, at<h16>(), st, at<int32_t>(), nullptr, seqs, T, T, Hq, Hkv, 128, 128,
                           scale, 1, at<h16>(), st, nullptr, at<void>(128), 0, nullptr);
}

static k3moe_status tree(int32_t seqs, int32_t T, int32_t Hq, int32_t width, int32_t page, int64_t st, size_t bytes)
{
    const k3moe_pages c{at<void>(), at<void>(), nullptr, nullptr, INT32_MAX, page};
    return k3moe_tree_attention(at<h16>(), st, &c, at<int32_t>(), width, at<int32_t>(), at<int32_t>(), nullptr, seqs, T, 64, Hq, 1,
                                128, 128, 1.0f, at<h16>(), st, nullptr, at<void>(), bytes, nullptr);
}

static k3moe_status lp(int32_t T, int32_t V, int32_t k, int64_t st, size_t bytes)
{
    return k3moe_logprobs(at<void>(), 1, st, T, V, nullptr, 0, nullptr, at<float>(), k ? at<int32_t>() : nullptr,
                          k ? at<float>() : nullptr, k, at<void>(), bytes, nullptr);
}

int main()
{
    const int32_t big = INT32_MAX;
    const k3moe_pages ok{at<void>(), at<void>(), nullptr, nullptr, big, 1 << 20}, odd{at<void>(), at<void>(), nullptr, nullptr, 1, 24};
    EXPECT(heads(0, 8, 64, 512, 64, 1e-5f, &ok), K3MOE_OK);
    EXPECT(heads(-1, 8, 64, 512, 64, 1e-5f, &ok), K3MOE_E_INVALID_ARG);
    EXPECT(heads(2, 8, 64, INT64_MIN, 64, 1e-5f, &ok), K3MOE_E_INVALID_ARG);
    EXPECT(heads(2, 8, 64, 512, INT32_MIN, 1e-5f, &ok), K3MOE_E_INVALID_ARG);
    EXPECT(heads(2, 8, 64, 512, 64, NAN, &ok), K3MOE_E_INVALID_ARG);
    EXPECT(heads(2, big, big, INT64_MAX, 64, 1e-5f, &ok), K3MOE_E_UNSUPPORTED_SHAPE);
    EXPECT(heads(big, 8, 64, 512, 64, 1e-5f, &ok), K3MOE_E_UNSUPPORTED_SHAPE);
    EXPECT(heads(2, 8, 64, 512, 64, 1e-5f, &odd), K3MOE_E_UNSUPPORTED_SHAPE);
    EXPECT(heads(2, 8, 64, 512, 64, 1e-5f, &ok), K3MOE_E_ALIGNMENT);   // q_out off by two bytes

    EXPECT(att(0, big, 8, 8, 1024, 1.0f, 0), K3MOE_OK);
    EXPECT(att(big, big, big, 1, 1024, 1.0f, 0), K3MOE_E_INVALID_ARG);     // heads wider than the rows
    EXPECT(att(big, big, 8, 8, INT64_MAX, 1.0f, 0), K3MOE_E_UNSUPPORTED_SHAPE);
    EXPECT(att(big, big, 8, 8, 1024, 1.0f, 0), K3MOE_E_UNSUPPORTED_SHAPE);
    EXPECT(att(1, 5, 8, 3, 1024, 1.0f, 0), K3MOE_E_INVALID_ARG);
    EXPECT(att(1, 5, 8, 8, 1024, -INFINITY, 0), K3MOE_E_INVALID_ARG);
    EXPECT(att(1, 5, 8, 8, 1024, 1.0f, 4), K3MOE_E_ALIGNMENT);
    EXPECT(att(1, 5, 8, 8, 1024, 1.0f, 0), K3MOE_E_WORKSPACE);             // misaligned

    size_t n = 0;
    EXPECT(k3moe_attention_workspace_size(big, big, big, big, 128, &n), K3MOE_OK);
    EXPECT(k3moe_attention_workspace_size(1, 1, big, 1, 128, &n), K3MOE_OK);
    EXPECT(k3moe_attention_workspace_size(0, 0, 0, big, 64, &n), K3MOE_OK);
    EXPECT(k3moe_attention_workspace_size(INT32_MIN, 1, 1, 1, 64, &n), K3MOE_E_INVALID_ARG);
    EXPECT(k3moe_tree_attention_workspace_size(4096, 1, 128, 64, &n), K3MOE_OK);
    EXPECT(k3moe_tree_attention_workspace_size(big, 1, 128, 64, &n), K3MOE_E_UNSUPPORTED_SHAPE);
    EXPECT(k3moe_tree_attention_workspace_size(INT32_MIN, -1, 128, 64, &n), K3MOE_E_INVALID_ARG);
    EXPECT(tree(1, 5, 8, 4, 64, 1024, n - 1), K3MOE_E_WORKSPACE);
    EXPECT(tree(0, 5, 8, 4, 64, 1024, 0), K3MOE_OK);
    EXPECT(tree(1, 5, 8, big, 1 << 20, 1024, n), K3MOE_E_UNSUPPORTED_SHAPE);
    EXPECT(tree(1, 5, 8, 4, INT32_MIN, 1024, n), K3MOE_E_INVALID_ARG);
    EXPECT(tree(1, 5, 8, 4, big, 1024, n), K3MOE_E_UNSUPPORTED_SHAPE);
    EXPECT(tree(big, big, 4096, 4, 64, 1 << 20, n), K3MOE_E_UNSUPPORTED_SHAPE);

    EXPECT(k3moe_logprobs_workspace_size(big, 1 << 24, 64, &n), K3MOE_E_UNSUPPORTED_SHAPE);
    EXPECT(k3moe_logprobs_workspace_size(big, big, 64, &n), K3MOE_E_UNSUPPORTED_SHAPE);
    EXPECT(k3moe_logprobs_workspace_size(1000, 163840, 64, &n), K3MOE_OK);
    EXPECT(lp(1000, 163840, 64, 163840, n - 1), K3MOE_E_WORKSPACE);
    EXPECT(lp(1000, 163840, 64, INT64_MIN, n), K3MOE_E_INVALID_ARG);
    EXPECT(lp(INT32_MIN, 163840, 64, 163840, n), K3MOE_E_INVALID_ARG);
    EXPECT(lp(0, 163840, 0, 0, 0), K3MOE_OK);
    if (failures) return 1;
    std::puts("ok");
    return 0;
}
