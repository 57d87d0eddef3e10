"""MI355X-native ZeRO / FSDP shard-local update.

The compute path is the C-ABI library libzero_shard.so (hand-written HIP
kernels for gfx950, declared in include/zero_shard.h); this package only
exposes it to Python.
"""
from .binding import (ACC_EMIT_BF16, ACC_NO_STORE, ACC_OVERWRITE, ACT8_BLOCK, DTYPE_BF16,
                      DTYPE_F32, GRAD_COMPACT, GRAD_FLAT, OUT_AG_SLOT, OUT_SHARD, AdamW, Layout,
                      Moments8, Rotation, ZeroError, load, zero_act8_pack, zero_act8_unpack,
                      zero_bias_grad, zero_bucket_pack, zero_embedding_grad,
                      zero_embedding_lookup, zero_gather_params, zero_grad_accumulate,
                      zero_head_norm_rotate, zero_head_norm_rotate_grad, zero_linear,
                      zero_linear_grad, zero_linear_input_grad, zero_moments8_pack,
                      zero_moments8_unpack, zero_reshard, zero_rms_norm, zero_rms_norm_grad,
                      zero_shard_step, zero_shard_step_accumulate, zero_shard_step_buckets,
                      zero_shard_step_moments8, zero_step_scalars)

__all__ = ["ACC_EMIT_BF16", "ACC_NO_STORE", "ACC_OVERWRITE", "ACT8_BLOCK", "DTYPE_BF16",
           "DTYPE_F32", "GRAD_COMPACT", "GRAD_FLAT", "OUT_AG_SLOT", "OUT_SHARD", "AdamW",
           "Layout", "Moments8", "Rotation", "ZeroError", "load", "zero_act8_pack",
           "zero_act8_unpack", "zero_bias_grad", "zero_bucket_pack", "zero_embedding_grad",
           "zero_embedding_lookup", "zero_gather_params", "zero_grad_accumulate",
           "zero_head_norm_rotate", "zero_head_norm_rotate_grad", "zero_linear",
           "zero_linear_grad", "zero_linear_input_grad", "zero_moments8_pack",
           "zero_moments8_unpack", "zero_reshard", "zero_rms_norm", "zero_rms_norm_grad",
           "zero_shard_step", "zero_shard_step_accumulate", "zero_shard_step_buckets",
           "zero_shard_step_moments8", "zero_step_scalars"]
