"""GB300-native NVFP4 W4A16 mixture-of-experts layer.

The layer runs in hand-written sm_103a CUDA kernels behind a C-ABI shared library
(``include/qmoe.h``, ``_lib/libqmoe.so``); ``qmoe`` is its thin ctypes binding.
"""

from .qmoe import (  # noqa: F401
    NVFP4MoE, QmoeError, moe_nvfp4_forward, moe_nvfp4_repack, moe_route, qmoe_forward_workspace_size,
    qmoe_max_tiles, qmoe_read_error, qmoe_repacked_fp4_size, qmoe_repacked_scale_size,
    qmoe_route_workspace_size, qmoe_sched_tile_n, qmoe_selftest_dequant, qmoe_selftest_timeout,
    QMOE_SCHED_AUTO, QMOE_SCHED_DECODE, QMOE_SCHED_PREFILL, QMOE_SCHED_PREFILL_PAIR, QMOE_W13,
    QMOE_W2, QMOE_SCALES_PLAIN, QMOE_SCALES_SWIZZLED_128X4)
from .operators import (  # noqa: F401
    moe_gate, moe_gate_backward, moe_sort_tokens, moe_sort_tokens_backward, moe_unsort_tokens,
    moe_unsort_tokens_backward, qmoe_default_read_error, qmoe_lora_linear,
    qmoe_lora_workspace_size, qmoe_sort_workspace_size, QMOE_DTYPE_BF16, QMOE_DTYPE_FP16,
    QMOE_DTYPE_FP32, QMOE_GATE_SIGMOID, QMOE_GATE_SOFTMAX)
from .block import (  # noqa: F401
    qmoe_block_norm, qmoe_block_norm_backward, qmoe_checkpoint8, qmoe_checkpoint8_restore,
    qmoe_gated_ffn, qmoe_gated_ffn_backward, qmoe_gated_ffn_backward_workspace_size,
    qmoe_gated_ffn_saved, qmoe_gated_ffn_workspace_size, QMOE_ACT_GELU, QMOE_ACT_SILU,
    QMOE_GATING_LINEAR, QMOE_GATING_SIGMOID)
