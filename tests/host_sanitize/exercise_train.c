/* Host-side checks of muonstep_train.h under AddressSanitizer and
 * UndefinedBehaviorSanitizer, without a GPU: calls that fail validation, that only
 * size a workspace, or that validate and plan and then fail at their first
 * launch.  Device pointers are fake, distinct addresses; nothing dereferences
 * them on the host.
 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "muonstep_train.h"

static int failures = 0;
#define EXPECT(cond)                                                                                                 \
    do {                                                                                                             \
        if (!(cond)) {                                                                                               \
            fprintf(stderr, "FAIL %s:%d: %s (last error: %s)\n", __FILE__, __LINE__, #cond, muon_last_error());      \
            ++failures;                                                                                              \
        }                                                                                                            \
    } while (0)

/* 8 TiB apart: more than the largest buffer of the sizes below */
#define AT(k) ((void*)(((uintptr_t)1 << 44) + ((uintptr_t)(k) << 43)))

static head_loss_t problem(int64_t tokens, int64_t vocab, int64_t dim, int grads) {
    head_loss_t p;
    memset(&p, 0, sizeof(p));
    p.hidden = AT(0);
    p.weight = AT(1);
    p.targets = AT(2);
    p.nll = AT(3);
    p.lse = AT(4);
    if (grads) {
        p.loss = AT(5);
        p.grad_hidden = AT(6);
        p.grad_weight = AT(7);
    }
    p.tokens = tokens;
    p.vocab = vocab;
    p.dim = p.hidden_stride = p.weight_stride = p.grad_hidden_stride = p.grad_weight_stride = dim;
    p.ignore_index = -100;
    return p;
}

static void head(void) {
    static const int64_t sizes[][3] = {{0, 1, 1}, {1, 1, 1}, {1, 8192, 512}, {33, 1000, 7}, {64, 131072, 2048},
        {2048, 4096, 512}, {1531, 12345, 600}, {16384, 8192, 512}, {8192, 131072, 2048}, {100000, 200000, 64},
        {1 << 24, 1 << 22, 65536}, {1 << 24, 1, 1}};
    for (size_t i = 0; i < sizeof(sizes) / sizeof(sizes[0]); ++i)
        for (int grads = 0; grads < 2; ++grads)
            for (int dtype = 0; dtype < 2; ++dtype) {
                head_loss_t p = problem(sizes[i][0], sizes[i][1], sizes[i][2], grads);
                p.dtype = dtype;
                p.softcap = dtype ? 30.0f : 0.0f;
                const size_t need = head_loss_workspace_size(&p);
                EXPECT(need > 0);
                EXPECT(head_loss(&p, AT(9), need - 1, NULL) == MUON_ERR_WORKSPACE);
                EXPECT(head_loss(&p, (char*)AT(9) + 8, need, NULL) == MUON_ERR_INVALID_ARG);
                if (sizes[i][0] > 0 && sizes[i][0] <= 16384)   /* validates, plans, then finds no device */
                    EXPECT(head_loss(&p, AT(9), need, NULL) == MUON_ERR_HIP);
                p.hidden = (char*)p.hidden + 2;                /* packed */
                EXPECT(head_loss_workspace_size(&p) > 0);
            }
    head_loss_t p = problem(10, 10, 8, 1);
    p.grad_weight_stride = 7;
    EXPECT(head_loss_workspace_size(&p) == 0);
    EXPECT(head_loss(NULL, AT(9), 1 << 20, NULL) == MUON_ERR_INVALID_ARG);
    EXPECT(head_loss_workspace_size(NULL) == 0);
}

static void adamw8(void) {
    static adamw8_tensor_t t[MUON_MAX_TENSORS];
    for (int i = 0; i < MUON_MAX_TENSORS; ++i) {
        char* b = (char*)AT(0) + ((uintptr_t)i << 24);
        memset(&t[i], 0, sizeof(t[i]));
        t[i].param = (float*)b;
        t[i].grad = b + (1 << 20);
        t[i].exp_avg = b + (2 << 20);
        t[i].rms = b + (3 << 20);
        if (i % 3) {
            t[i].exp_avg_scale = (float*)(b + (4 << 20));
            t[i].rms_scale = (float*)(b + (5 << 20));
        }
        t[i].ema = i % 2 ? (float*)(b + (6 << 20)) : NULL;
        t[i].copy = i % 5 ? b + (7 << 20) : NULL;
        t[i].grad_bf16 = i % 2;
        t[i].numel = i % 7 ? 1 + 37 * i : 0;
    }
    static const int counts[] = {1, 2, 8, 9, 192, 193, 400, MUON_MAX_TENSORS};
    for (size_t i = 0; i < sizeof(counts) / sizeof(counts[0]); ++i) {
        const int rc = adamw8_step(t, counts[i], 1e-3f, 0.9f, 0.999f, 1e-8f, 0.01f, 3, 0.9f, 1, ~(uint64_t)0, NULL);
        EXPECT(rc == (counts[i] == 1 ? MUON_OK : MUON_ERR_HIP));       /* the first tensor is empty: nothing to launch */
    }
    EXPECT(adamw8_step(t, 2, NAN, 0.9f, 0.999f, 1e-8f, 0.01f, 3, 0.9f, 0, 0, NULL) == MUON_ERR_INVALID_ARG);
    t[2].param = t[1].param;
    EXPECT(adamw8_step(t, 4, 1e-3f, 0.9f, 0.999f, 1e-8f, 0.01f, 3, 0.9f, 0, 0, NULL) == MUON_ERR_UNSUPPORTED);
    t[1].numel = INT64_MAX;
    EXPECT(adamw8_step(t, 2, 1e-3f, 0.9f, 0.999f, 1e-8f, 0.01f, 3, 0.9f, 0, 0, NULL) == MUON_ERR_UNSUPPORTED);
    EXPECT(adamw8_encode(AT(0), AT(1), AT(2), AT(3), AT(4), AT(5), 1000, NULL) == MUON_ERR_HIP);
    EXPECT(adamw8_decode(AT(0), AT(1), AT(2), AT(3), AT(4), AT(5), INT64_MAX, NULL) == MUON_ERR_UNSUPPORTED);
}

int main(void) {
    head();
    adamw8();
    if (failures) return 1;
    printf("ALL OK\n");
    return 0;
}
