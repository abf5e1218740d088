/* Host-side checks of muonstep_linear8.h under AddressSanitizer and
 * UndefinedBehaviorSanitizer, without a GPU: calls that fail validation, that only
 * size a workspace, or that validate and plan and then fail at their first
 * launch.  Device pointers are fake, distinct addresses; nothing dereferences
 * them on the host.
 */
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "muonstep_linear8.h"

static int failures = 0;
#define EXPECT(cond)                                                                                                 \
    do {                                                                                                             \
        if (!(cond)) {                                                                                               \
            fprintf(stderr, "FAIL %s:%d: %s (last error: %s)\n", __FILE__, __LINE__, #cond, muon_last_error());      \
            ++failures;                                                                                              \
        }                                                                                                            \
    } while (0)

/* 32 TiB apart: more than the largest buffer of the sizes below */
#define AT(k) ((void*)(((uintptr_t)1 << 46) + ((uintptr_t)(k) << 45)))

static blocks8_t coded(int k, int64_t dim) {
    blocks8_t b = {AT(k), AT(k + 1), (dim + 15) / 16 * 16, (dim + 511) / 512 * 4};
    return b;
}

/* A size that validates and launches (and finds no device), one that does nothing, or one that is refused. */
static int expected(int64_t rows, int refused) { return refused ? refused : rows == 0 ? MUON_OK : MUON_ERR_HIP; }

int main(void) {
    static const int64_t sizes[] = {0, 1, 2, 15, 16, 17, 33, 64, 127, 129, 1000, 4097, 1 << 14, 1 << 17, 1 << 18, (1 << 18) + 1,
                                    1 << 24, (1 << 24) + 1, INT64_MAX, -1, INT64_MIN};
    const int n = (int)(sizeof(sizes) / sizeof(sizes[0]));
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < n; ++j) {
            const int64_t rows = sizes[i], dim = sizes[j];
            const int bad = dim < 1 || rows < 0 ? MUON_ERR_INVALID_ARG
                            : rows > MUON_LINEAR8_MAX_ROWS || dim > MUON_LINEAR8_MAX_DIM ? MUON_ERR_UNSUPPORTED : 0;
            const int64_t d = bad ? 128 : dim;
            for (int act = 0; act < 4; ++act)
                for (int type = 0; type < 3; ++type) {
                    act8_encode_t e;
                    memset(&e, 0, sizeof(e));
                    e.x = AT(0); e.rows = rows; e.dim = dim; e.x_stride = d; e.dtype = type; e.activation = act;
                    e.codes = coded(1, d);
                    if (act) e.out = coded(3, d);
                    EXPECT(act8_encode(&e, NULL) == expected(rows, bad));
                    act8_backward_t b;
                    memset(&b, 0, sizeof(b));
                    b.u = coded(0, d); b.grad = AT(2); b.out = AT(2 + act % 2); b.rows = rows; b.dim = dim;
                    b.grad_stride = b.out_stride = d; b.dtype = type; b.activation = act;
                    b.out8 = coded(4, d);
                    EXPECT(act8_backward(&b, NULL) == (act || bad ? expected(rows, bad) : MUON_ERR_INVALID_ARG));
                }
            const blocks8_t q = coded(0, d);
            EXPECT(act8_decode(&q, j % 2, rows, dim, AT(2), d, i % 3, NULL) == expected(rows, bad));
            for (int k = 0; k < n; ++k) {
                const int64_t cols = sizes[k];
                const int refused = bad == MUON_ERR_INVALID_ARG || cols < 1 ? MUON_ERR_INVALID_ARG
                                    : bad || cols > MUON_LINEAR8_MAX_DIM ? MUON_ERR_UNSUPPORTED : 0;
                const int64_t c = refused ? 128 : cols;
                matmul8_t m;
                memset(&m, 0, sizeof(m));
                m.a = coded(0, d); m.b = coded(2, d); m.y = AT(4); m.rows = rows; m.cols = cols; m.dim = dim; m.y_stride = c;
                size_t need = matmul8_workspace_size(&m);
                if (refused) EXPECT(need == 0 && matmul8(&m, AT(6), 1 << 20, NULL) == refused);
                else if (need) EXPECT(matmul8(&m, AT(6), need, NULL) == expected(rows, 0) && matmul8(&m, AT(6), need - 1, NULL) == MUON_ERR_WORKSPACE);
                else EXPECT(matmul8(&m, AT(6), 1 << 20, NULL) == MUON_ERR_UNSUPPORTED);      /* too many tiles */
                act8_grad_weight_t g;
                memset(&g, 0, sizeof(g));
                g.x = coded(0, d); g.grad = AT(2); g.out = AT(3); g.rows = rows; g.cols = cols; g.dim = dim; g.grad_stride = c;
                g.out_stride = d; g.accumulate = i % 2;
                need = act8_grad_weight_workspace_size(&g);
                if (refused) EXPECT(need == 0 && act8_grad_weight(&g, AT(6), 1 << 20, NULL) == refused);
                else if (need) EXPECT(act8_grad_weight(&g, AT(6), need, NULL) == (rows == 0 && g.accumulate ? MUON_OK : MUON_ERR_HIP));
                else EXPECT(act8_grad_weight(&g, AT(6), 1 << 20, NULL) == MUON_ERR_UNSUPPORTED);
                weight8_encode_t w;
                memset(&w, 0, sizeof(w));
                w.weight = AT(0); w.rows = cols; w.dim = dim; w.weight_stride = d; w.dtype = k % 3;
                w.codes = coded(1, d);
                if (k % 2) w.transposed = coded(3, c);
                if (rows == 1) {
                    const int rc = weight8_encode(&w, NULL);
                    EXPECT(rc == (refused ? refused : MUON_ERR_HIP) || (!refused && rc == MUON_ERR_UNSUPPORTED));
                }
            }
        }
    EXPECT(act8_encode(NULL, NULL) == MUON_ERR_INVALID_ARG && act8_backward(NULL, NULL) == MUON_ERR_INVALID_ARG);
    EXPECT(weight8_encode(NULL, NULL) == MUON_ERR_INVALID_ARG && matmul8(NULL, NULL, 0, NULL) == MUON_ERR_INVALID_ARG);
    EXPECT(act8_grad_weight(NULL, NULL, 0, NULL) == MUON_ERR_INVALID_ARG && act8_decode(NULL, 0, 1, 1, NULL, 1, 0, NULL) == MUON_ERR_INVALID_ARG);
    if (failures) return 1;
    printf("ALL OK\n");
    return 0;
}
