/* A plain C99 caller of the adapter and checkpoint entry points of include/q8.h: the header's own
 * types, and arguments that the host-side checks decide.  Built and run by
 * test_lora_host.py. */
#include <stdio.h>

#include "q8.h"

static int fails = 0;

static void expect(const char* what, q8_status got, q8_status want) {
    if (got != want) {
        printf("%s: got %d (%s), want %d\n", what, (int)got, q8_status_string(got), (int)want);
        ++fails;
    }
}

int main(void) {
    q8_adapters ad;
    q8_saved_input in;
    ad.a = NULL;
    ad.b = NULL;
    ad.scale = NULL;
    ad.count = 4;
    ad.rank = 16;
    in.x = NULL;
    in.exps = NULL;
    in.group = 0;
    expect("lora", q8_linear_w8a16_lora(NULL, NULL, NULL, NULL, &ad, NULL, NULL, Q8_BF16, NULL, 1, 16,
                                        64, NULL, 0, NULL), Q8_ERR_NULL);
    expect("lora M = 0", q8_linear_w8a16_lora(NULL, NULL, NULL, NULL, &ad, NULL, NULL, Q8_F32, NULL,
                                              0, 16, 64, NULL, 0, NULL), Q8_OK);
    ad.rank = 12;
    expect("lora rank", q8_linear_w8a16_lora(NULL, NULL, NULL, NULL, &ad, NULL, NULL, Q8_BF16, NULL,
                                             1, 16, 64, NULL, 0, NULL), Q8_ERR_ARG);
    ad.rank = 16;
    expect("backward", q8_linear_w8a16_lora_backward(NULL, NULL, NULL, &ad, NULL, NULL, &in, NULL,
                                                     NULL, NULL, 0, 1, 16, 64, NULL, 0, NULL), Q8_OK);
    expect("backward N", q8_linear_w8a16_lora_backward(NULL, NULL, NULL, &ad, NULL, NULL, &in, NULL,
                                                       NULL, NULL, 0, 1, 15, 64, NULL, 0, NULL),
           Q8_ERR_SHAPE);
    expect("save", q8_checkpoint_save(NULL, Q8_BF16, 1, 64, 48, NULL, NULL, NULL), Q8_ERR_ARG);
    expect("load", q8_checkpoint_load(NULL, NULL, 32, NULL, Q8_F32, 1, 64, NULL), Q8_ERR_NULL);
    expect("wgrad", q8_checkpoint_wgrad(NULL, NULL, NULL, 32, NULL, 0, 1, 16, 64, NULL, 0, NULL),
           Q8_ERR_NULL);
    if (q8_workspace_bytes(Q8_OP_LINEAR_W8A16_LORA, 40, 32, 64, 16) == 0) ++fails;
    if (q8_workspace_bytes(Q8_OP_LINEAR_W8A16_LORA_BACKWARD, 4, 32, 64, 16) == 0) ++fails;
    if (q8_workspace_bytes(Q8_OP_CHECKPOINT_WGRAD, 4, 32, 64, 0) != 0) ++fails;
    printf("failures: %d\n", fails);
    return fails == 0 ? 0 : 1;
}
