/* include/carbon_lm.h from C: compiles as C99 and answers argument errors,
 * empty problems and workspace queries without a GPU. */
#include "carbon_lm.h"

#include <stdio.h>

#define CHECK(cond)                                        \
    do {                                                   \
        if (!(cond)) {                                     \
            fprintf(stderr, "line %d: %s\n", __LINE__, #cond); \
            return 1;                                      \
        }                                                  \
    } while (0)

int main(void) {
    char buf[64];
    void *p = buf;
    CHECK(carbon_embedding_fwd(NULL, NULL, NULL, 0, 3, 4, 1.0f, CARBON_BF16, NULL) == CARBON_OK);
    CHECK(carbon_embedding_fwd(p, p, NULL, 2, 3, 4, 1.0f, CARBON_BF16, NULL) == CARBON_ERR_INVALID_ARG);
    CHECK(carbon_embedding_bwd(NULL, NULL, NULL, 0, 0, 4, 1.0f, -1, 0, NULL, 0, CARBON_F32, NULL) == CARBON_OK);
    CHECK(carbon_embedding_bwd(p, p, NULL, 2, 3, 4, 1.0f, 3, 0, p, 64, CARBON_F32, NULL) == CARBON_ERR_INVALID_ARG);
    CHECK(carbon_rms_norm_fwd(p, NULL, NULL, NULL, NULL, p, NULL, p, 2, 4, -1.0f, CARBON_F16, NULL) == CARBON_ERR_INVALID_ARG);
    CHECK(carbon_rms_norm_bwd(NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, 0, 4, NULL, 0, CARBON_F16, NULL) ==
          CARBON_OK);
    CHECK(carbon_rms_norm_expand(p, NULL, NULL, NULL, 1, 1, CARBON_F16, NULL) == CARBON_ERR_INVALID_ARG);
    CHECK(carbon_linear_xent_fwd(NULL, NULL, NULL, NULL, NULL, NULL, NULL, 4, 8, 16, -100, CARBON_REDUCE_MEAN, NULL, 0,
                                 CARBON_F32, NULL) == CARBON_ERR_UNSUPPORTED);
    CHECK(carbon_linear_xent_bwd(NULL, NULL, NULL, NULL, NULL, NULL, NULL, 4, 12, 16, -100, CARBON_REDUCE_SUM, NULL, 0,
                                 CARBON_BF16, NULL) == CARBON_ERR_INVALID_ARG);
    CHECK(carbon_embedding_bwd_workspace(100, 10, 8) > 0);
    CHECK(carbon_rms_norm_bwd_workspace(100, 8) > 0);
    CHECK(carbon_linear_xent_fwd_workspace(100, 8, 10) > 0);
    CHECK(carbon_linear_xent_bwd_workspace(100, 8, 10) > carbon_linear_xent_fwd_workspace(1, 8, 10));
    CHECK(carbon_linear_xent_bwd_workspace(-1, 8, 10) == -1);
    puts("ok");
    return 0;
}
