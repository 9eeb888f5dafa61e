/* The calls of a block's dense side from plain C99: size queries and argument checks, which need no
 * GPU.  Prints one line per failed check; exit code = failures. */
#include <math.h>
#include <stdio.h>

#include "qmoe.h"

static int fails = 0;
#define CHECK(cond)                                          \
  do {                                                       \
    if (!(cond)) {                                           \
      printf("FAIL %s:%d %s\n", __FILE__, __LINE__, #cond);  \
      ++fails;                                               \
    }                                                        \
  } while (0)

int main(void) {
  CHECK(qmoe_gated_ffn_workspace_size(16, 7168, 2048) > (size_t)16 * 2048 * 2);
  CHECK(qmoe_gated_ffn_workspace_size(16, 7168, 2044) == 0);
  CHECK(qmoe_gated_ffn_backward_workspace_size(16, 7168, 2048, 8) >
        qmoe_gated_ffn_backward_workspace_size(16, 7168, 2048, 16));
  CHECK(qmoe_gated_ffn_backward_workspace_size(16, 7168, 2048, 4) == 0);
  CHECK(qmoe_block_norm_backward_workspace_size(16, 7168) > 0);
  CHECK(qmoe_block_norm_backward_workspace_size(16, 0) == 0);
  CHECK(qmoe_block_norm(NULL, QMOE_DTYPE_BF16, 8, NULL, 0, 1.0f, NULL, QMOE_DTYPE_BF16,
                        QMOE_GATE_TOKEN, 1, QMOE_GATING_LINEAR, NULL, NULL, QMOE_DTYPE_FP32, 0.0f,
                        1e-6f, 0, 8, NULL, NULL, NULL, NULL, NULL) == QMOE_OK);
  CHECK(qmoe_block_norm(NULL, QMOE_DTYPE_BF16, 7, NULL, 0, 1.0f, NULL, QMOE_DTYPE_BF16,
                        QMOE_GATE_TOKEN, 1, QMOE_GATING_LINEAR, NULL, NULL, QMOE_DTYPE_FP32, 0.0f,
                        1e-6f, 4, 8, NULL, NULL, NULL, NULL, NULL) == QMOE_ERR_SHAPE);
  CHECK(qmoe_checkpoint8(NULL, QMOE_DTYPE_FP16, 32, 4, 32, NULL, NULL, NULL) == QMOE_ERR_ARG);
  CHECK(qmoe_checkpoint8_restore(NULL, NULL, 9, 4, 32, NULL, NULL) == QMOE_ERR_ARG);
  CHECK(qmoe_gated_ffn(NULL, QMOE_DTYPE_BF16, 64, NULL, NULL, QMOE_ACT_GELU, INFINITY, 0, 64, 128,
                       NULL, NULL, NULL, NULL, 0, NULL) == QMOE_OK);
  CHECK(qmoe_gated_ffn(NULL, QMOE_DTYPE_FP32, 64, NULL, NULL, QMOE_ACT_SILU, INFINITY, 4, 64, 128,
                       NULL, NULL, NULL, NULL, 0, NULL) == QMOE_ERR_ARG);
  CHECK(qmoe_gated_ffn_backward(NULL, QMOE_DTYPE_BF16, 64, NULL, 64, NULL, NULL, NULL, NULL, NULL,
                                QMOE_ACT_SILU, -1.0f, 4, 64, 128, NULL, NULL, NULL, NULL, 0,
                                NULL) == QMOE_ERR_ARG);
  printf("%s: %d failure(s)\n", fails ? "FAILED" : "ok", fails);
  return fails;
}
