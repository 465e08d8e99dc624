"""GB300-native ZeRO sharded mixed-precision optimizer step.

The compute lives in libzero.so (C ABI: include/zero.h; CUDA kernels for
sm_103a in csrc/); this package is its Python binding.  ``engine`` wires a
model's backward pass into it; ``train_ops`` holds the operators of a
training step around it (gradient norm and clipping, block join, expert
routing and permutation, token embedding, cross entropy over the vocabulary);
``workloads`` holds the seeded synthetic parameter groups used
by the tests and the benchmark.
"""
from .zero import (AMP_STATE_BYTES, ZERO_BF16, ZERO_FP16, ZERO_PART_FLAT,  # noqa: F401
                   ZERO_PART_ROUND_ROBIN, ZERO_REDUCE_AVG, ZERO_REDUCE_SUM, AdamW, AmpConfig,
                   AmpState, FloorProbe, Plan, ReduceScatterBucketAmp, ReduceScatterRange,
                   Zero3Pass, ZeroError, ZeroStep,
                   amp_state_tensor, lib, read_amp_state, zero_adamw_shard_step, zero_allgather,
                   zero_amp_init, zero_amp_workspace_bytes, zero_cpu_adamw_shard_step,
                   zero_init_shards, zero_last_error, zero_launch_count, zero_memory_bytes,
                   zero_offload_step, zero_offload_step_amp,
                   zero_plan_describe, zero_plan_destroy, zero_plan_info, zero_plan_partitions,
                   zero_plan_segments, zero_plan_shard, zero_plan_total, zero_reduce_scatter,
                   zero_reduce_scatter_bucket_amp, zero_reduce_scatter_range,
                   zero_floor_probe, zero_selftest_wait_timeout, zero_step, zero_step_amp,
                   zero_step_amp_noalloc, zero_step_amp_reduced, zero_step_amp_shards,
                   zero_sync, zero_version, zero_zero3_pass)


_TRAIN_OPS = ("ClipGradNorm", "CrossEntropy", "ExpertOrder", "ExpertRoute", "GradNorm",
              "NormResult", "block_join", "embedding", "expert_combine", "expert_dispatch",
              "expert_route", "linear_cross_entropy", "read_norm_result", "zero_block_join",
              "zero_block_join_backward", "zero_block_join_workspace_bytes",
              "zero_clip_grad_norm", "zero_embedding", "zero_embedding_backward",
              "zero_embedding_workspace_bytes", "zero_expert_combine",
              "zero_expert_combine_backward", "zero_expert_dispatch",
              "zero_expert_dispatch_backward", "zero_expert_route", "zero_expert_route_backward",
              "zero_expert_route_workspace_bytes", "zero_expert_sort",
              "zero_expert_sort_workspace_bytes", "zero_grad_norm",
              "zero_grad_norm_workspace_bytes", "zero_linear_cross_entropy",
              "zero_linear_cross_entropy_backward", "zero_linear_cross_entropy_rest",
              "zero_linear_cross_entropy_rest_backward", "zero_linear_cross_entropy_workspace_bytes")


def __getattr__(name):
    # train_ops needs torch at import time, this package does not
    if name in _TRAIN_OPS:
        from . import train_ops
        value = getattr(train_ops, name)
        globals()[name] = value
        return value
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
