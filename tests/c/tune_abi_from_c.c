/* The operators of fine-tuning and scoring in include/carbon_lm.h from C: argument
 * errors, empty problems and workspace queries without a GPU. */
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
    void *p = buf, *out[1];
    const void *grads[1];
    int64_t sizes[1] = {0};
    int dtypes[1] = {CARBON_BF16};
    out[0] = p;
    grads[0] = p;
    CHECK(carbon_clip_grads(NULL, out, grads, sizes, dtypes, 1, 1.0f, 0.0f, NULL, 0, NULL) == CARBON_OK);
    CHECK(carbon_clip_grads(NULL, NULL, grads, sizes, dtypes, 1, 1.0f, 0.0f, NULL, 0, NULL) == CARBON_ERR_INVALID_ARG);
    CHECK(carbon_clip_grads_workspace(sizes, 1) > 0);
    CHECK(carbon_linear_logp_fwd(NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, 4, 8, 16, 0, 1.0f, -100, NULL, 0,
                                 CARBON_F32, NULL) == CARBON_ERR_UNSUPPORTED);
    CHECK(carbon_linear_logp_bwd(NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, 4, 8, 16, 0.0f, -100, NULL, 0,
                                 CARBON_BF16, NULL) == CARBON_ERR_INVALID_ARG);
    CHECK(carbon_linear_logp_fwd_workspace(300, 8, 100, 5) > carbon_linear_logp_fwd_workspace(300, 8, 100, 0));
    CHECK(carbon_linear_logp_fwd_workspace(300, 8, 100, 29) == -1);
    CHECK(carbon_linear_logp_bwd_workspace(300, 8, -1) == -1);
    CHECK(carbon_lora_linear_fwd(NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, 0, 8, 8, 1, 8, NULL, 0, CARBON_F16,
                                 NULL) == CARBON_OK);
    CHECK(carbon_lora_linear_fwd(NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, 4, 8, 8, 1, 8, NULL, 0, CARBON_F16,
                                 NULL) == CARBON_ERR_INVALID_ARG);
    CHECK(carbon_lora_linear_bwd(NULL, NULL, p, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, 4, 8, 8, 1, 8, NULL, 0,
                                 CARBON_F16, NULL) == CARBON_ERR_INVALID_ARG);
    CHECK(carbon_lora_linear_u_elements(10, 24) == 10 * 3 * 32);
    CHECK(carbon_lora_linear_fwd_workspace(10, 8, 8, 2, 129) == -1);
    CHECK(carbon_lora_linear_bwd_workspace(5000, 64, 64, 2, 8) > carbon_lora_linear_fwd_workspace(5000, 64, 64, 2, 8));
    puts("ok");
    return 0;
}
