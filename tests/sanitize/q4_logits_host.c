/*
 * Drives the host side of the 4-bit linears and the operators on logits
 * (include/rbq.h) so that it can run under AddressSanitizer and
 * UndefinedBehaviorSanitizer: workspace sizes and plans over ordinary and
 * extreme shapes, where gradients may lie, and argument checks.  No call here
 * reaches a device; the pointers are aligned stand-in addresses that the checks
 * compare but never dereference.
 * Test infrastructure: built and run by tests/test_sanitizers_q4_cpu.py.
 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "rbq.h"

static int failures = 0;
#define CHECK(cond)                                                     \
    do {                                                                \
        if (!(cond)) {                                                  \
            fprintf(stderr, "FAIL %s:%d: %s\n", __FILE__, __LINE__, #cond); \
            ++failures;                                                 \
        }                                                               \
    } while (0)
#define N(a) (sizeof(a) / sizeof((a)[0]))

static void *buf(int k) { return (void *)(((uintptr_t)1 << 40) + (uintptr_t)k * ((uintptr_t)1 << 20)); }
static void *odd(int k) { return (void *)((uintptr_t)buf(k) + 1); }

static const int32_t OUTS[] = {1, 15, 16, 255, 256, 257, 4096, 11008, 128256, 1 << 20, RBQ_Q4_MAX_FEATURES};
static const int32_t INS[] = {32, 96, 128, 160, 4096, 4128, 14336, 28704, 1 << 20, 1 << 23, (1 << 23) + 32, RBQ_Q4_MAX_FEATURES};
static const int32_t COUNTS[] = {1, 4, 5, 16, 17, 64, 65, 300, 2048, 100000, 1 << 24, INT32_MAX};
static const int32_t VOCABS[] = {1, 7, 8, 9, 1000, 32000, 47993, 48000, 50257, 128256, 1 << 20, RBQ_VOCAB_MAX};

static void sizes(void)
{
    for (size_t o = 0; o < N(OUTS); ++o)
        for (size_t i = 0; i < N(INS); ++i)
            for (size_t m = 0; m < N(COUNTS); ++m) {
                const size_t a = rbq_gemm_q4_workspace_bytes(OUTS[o], INS[i], COUNTS[m], RBQ_Y_F16);
                const size_t b = rbq_gemm_q4_workspace_bytes(OUTS[o], INS[i], COUNTS[m], RBQ_Y_F32);
                const size_t one = (size_t)4 * (size_t)OUTS[o] * (size_t)COUNTS[m];
                CHECK(a == b && a % one == 0 && a / one <= 16 && a != one);
            }
    for (size_t m = 0; m < N(COUNTS); ++m)
        for (size_t v = 0; v < N(VOCABS); ++v)
            for (int32_t k = 0; k <= RBQ_TOP_MAX; ++k) {
                const size_t rows = (size_t)COUNTS[m];
                const size_t a = rbq_token_logprobs_workspace_bytes(COUNTS[m], VOCABS[v], k);
                const size_t b = rbq_distill_workspace_bytes(COUNTS[m], VOCABS[v], k);
                CHECK(a % (rows * (16 + 8 * (size_t)k)) == 0 && a / (rows * (16 + 8 * (size_t)k)) <= 256);
                CHECK((a == 0) == (b == 0) && (b == 0 || (b - 4 * rows * (size_t)k) % (rows * 16) == 0));
            }
    const int32_t wild[] = {INT32_MIN, -1, 0, RBQ_VOCAB_MAX + 1, INT32_MAX};
    for (size_t i = 0; i < N(wild); ++i) {
        CHECK(rbq_token_logprobs_workspace_bytes(4, wild[i], 0) == 0 && rbq_distill_workspace_bytes(4, wild[i], 0) == 0);
        CHECK(wild[i] == 0 || rbq_token_logprobs_workspace_bytes(4, 200000, wild[i]) == 0);
        CHECK(wild[i] == 0 || rbq_distill_workspace_bytes(4, 200000, wild[i]) == 0);
        CHECK(wild[i] > 0 || rbq_token_logprobs_workspace_bytes(wild[i], 200000, 4) == 0);
        CHECK(wild[i] > 0 || rbq_gemm_q4_workspace_bytes(4096, 4096, wild[i], 0) == 0);
        CHECK(rbq_gemm_q4_workspace_bytes(4096, wild[i], 128, 0) == 0);
    }
    CHECK(rbq_gemm_q4_workspace_bytes(INT32_MAX, INT32_MAX - 31, INT32_MAX, 0) == 0);
    CHECK(rbq_gemm_q4_workspace_bytes(4096, 4096, 128, UINT32_MAX) == 0);
}

/* What a call says of a gradient's place beside its logits. */
static rbq_status place(int32_t M, int32_t vocab, int64_t stride, const void *d, int64_t d_stride)
{
    return rbq_distill_backward(buf(1), RBQ_L_F16, M, vocab, stride, 1.0f, NULL, NULL, 0, 0, odd(0), (void *)d, d_stride,
                                NULL, NULL, 0, NULL, NULL);
}

static void places(void)
{
    /* (d_loss at an odd address: what passes the check of the place is RBQ_ERR_ALIGNMENT) */
    char *x = buf(1);
    CHECK(place(4, 100, 100, x, 100) == RBQ_ERR_ALIGNMENT);
    CHECK(place(4, 100, 250, x + 200, 250) == RBQ_ERR_ALIGNMENT);
    CHECK(place(4, 100, 250, x + 300, 250) == RBQ_ERR_ALIGNMENT);
    const int64_t strides[] = {100, 101, 200, 250, (int64_t)1 << 31};
    for (size_t s = 0; s < N(strides); ++s)
        for (size_t e = 0; e < N(strides); ++e)
            for (size_t m = 0; m < N(COUNTS); ++m) {
                CHECK(place(COUNTS[m], 100, strides[s], x + 2, strides[e]) == RBQ_ERR_INVALID_ARG);
                CHECK(place(COUNTS[m], 100, strides[s], x - 2, strides[e]) == RBQ_ERR_INVALID_ARG);
            }
    CHECK(place(INT32_MAX, RBQ_VOCAB_MAX, (int64_t)1 << 31, x, (int64_t)1 << 31) == RBQ_ERR_ALIGNMENT);
    CHECK(place(4, 100, INT64_MAX, x, 100) == RBQ_ERR_UNSUPPORTED);
    CHECK(place(4, 100, 100, x, INT64_MAX) == RBQ_ERR_UNSUPPORTED);
    CHECK(place(4, 100, INT64_MIN, x, 100) == RBQ_ERR_INVALID_ARG);
    CHECK(place(4, 100, 100, x, INT64_MIN) == RBQ_ERR_INVALID_ARG);
}

static void arguments(void)
{
    const int32_t wild[] = {INT32_MIN, -1, 31, 33, INT32_MAX};
    for (size_t i = 0; i < N(wild); ++i) {
        CHECK(rbq_encode_q4(buf(0), 64, wild[i], buf(1), buf(2), NULL, NULL, NULL) == RBQ_ERR_INVALID_ARG);
        CHECK(rbq_gemm_q4(buf(0), buf(1), NULL, 64, wild[i], buf(2), 4, buf(3), 0, NULL, 0, NULL) == RBQ_ERR_INVALID_ARG);
    }
    CHECK(rbq_encode_q4(buf(0), INT32_MAX, 64, buf(1), buf(2), NULL, NULL, NULL) == RBQ_ERR_UNSUPPORTED);
    CHECK(rbq_encode_q4(odd(0), 64, 64, buf(1), buf(2), NULL, NULL, NULL) == RBQ_ERR_ALIGNMENT);
    CHECK(rbq_gemm_q4(buf(0), buf(1), NULL, 64, 64, buf(2), INT32_MIN, buf(3), 0, NULL, 0, NULL) == RBQ_ERR_INVALID_ARG);
    CHECK(rbq_gemm_q4(buf(0), buf(1), NULL, 64, 64, buf(2), 4, buf(3), 0, NULL, SIZE_MAX, NULL) == RBQ_ERR_INVALID_ARG);
    CHECK(rbq_gemm_q4(buf(0), odd(1), NULL, 64, 64, buf(2), 4, buf(3), 0, NULL, 0, NULL) == RBQ_ERR_ALIGNMENT);
    const float T[] = {0.0f, -1.0f, NAN, INFINITY, 1e-4f, 1e4f};
    for (size_t i = 0; i < N(T); ++i) {
        CHECK(rbq_token_logprobs(buf(0), 0, 4, 100, 100, T[i], buf(1), buf(2), NULL, 0, NULL, NULL, NULL, 0, NULL, NULL) ==
              RBQ_ERR_INVALID_ARG);
        CHECK(rbq_distill_forward(buf(0), 0, 4, 100, 100, T[i], NULL, NULL, 0, 0, buf(1), NULL, 0, NULL, NULL) ==
              RBQ_ERR_INVALID_ARG);
    }
    CHECK(rbq_token_logprobs(buf(0), UINT32_MAX, 4, 100, 100, 1.0f, buf(1), buf(2), NULL, 0, NULL, NULL, NULL, 0, NULL,
                             NULL) == RBQ_ERR_INVALID_ARG);
    CHECK(rbq_token_logprobs(buf(0), 0, INT32_MIN, 100, 100, 1.0f, buf(1), buf(2), NULL, 0, NULL, NULL, NULL, 0, NULL,
                             NULL) == RBQ_ERR_INVALID_ARG);
    CHECK(rbq_token_logprobs_backward(buf(0), 0, 4, 100, 100, 1.0f, NULL, buf(1), NULL, buf(2), 100, NULL, NULL, NULL, 0,
                                      NULL, NULL) == RBQ_ERR_INVALID_ARG);
    CHECK(rbq_distill_forward(buf(0), 0, 4, 100, 100, 1.0f, buf(1), NULL, 3, 0, buf(2), NULL, 0, NULL, NULL) ==
          RBQ_ERR_INVALID_ARG);
    CHECK(rbq_distill_forward(buf(0), 0, 4, 100, 100, 1.0f, buf(1), buf(2), 3, UINT32_MAX, buf(3), NULL, 0, NULL, NULL) ==
          RBQ_ERR_INVALID_ARG);
    /* nothing to do: no device is looked for */
    CHECK(rbq_encode_q4(NULL, 0, 64, NULL, NULL, NULL, NULL, NULL) == RBQ_OK);
    CHECK(rbq_gemm_q4(NULL, NULL, NULL, 64, 64, NULL, 0, NULL, 0, NULL, 0, NULL) == RBQ_OK);
    CHECK(rbq_distill_forward(NULL, 0, 0, 100, 100, 1.0f, NULL, NULL, 0, 0, NULL, NULL, 0, NULL, NULL) == RBQ_OK);
}

int main(void)
{
    sizes();
    places();
    arguments();
    if (failures != 0) {
        fprintf(stderr, "%d checks failed\n", failures);
        return 1;
    }
    puts("4-bit and logits host checks passed");
    return 0;
}
