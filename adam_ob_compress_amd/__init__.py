"""1-bit Adam (and 1-bit LAMB) optimizer step on AMD MI355X (gfx950): HIP kernels behind a C ABI
(libobadam.so).

Python side = argument marshalling (``_native``), host schedules (``schedule``) and the seeded
synthetic workloads (``synth``).  Importing the package does not load the library; the first call does,
and raises if it has not been built (there is no CPU fallback).
"""
from ._native import (  # noqa: F401
    KERNEL_NAMES, OB_BF16, OB_EF_EMA, OB_EF_PLAIN, OB_F16, OB_F32, OB_ROUND_NEAREST, OB_ROUND_STOCHASTIC,
    OB_KERNEL_CHUNK_SUMSQ,
    OB_KERNEL_COMPRESS, OB_KERNEL_DENSE, OB_KERNEL_DIAG, OB_KERNEL_LAMB_APPLY, OB_KERNEL_SERVER_APPLY,
    OB_KERNEL_SERVER_SUMSQ, OB_KERNEL_TRUST_RATIO, OB_KERNEL_UNPACK, LIB_PATH, ObError, Plan, hparams,
    OB_ERR_OOM, OB_ERR_SIZE, OB_NOALLOC_SCRATCH_BYTES,
    lib, ob_adam_compress_step, ob_adam_compress_step_noalloc, ob_adam_warmup_step, ob_adam_worker_compress,
    ob_adam_worker_update,
    ob_hparams, ob_lamb_compress_step, ob_lamb_worker_update,
    ob_lamb_warmup_step, ob_pack, ob_plan_create, ob_plan_read_timing, ob_plan_set_diagnostics,
    ob_plan_set_guard,
    ob_plan_set_timing,
    ob_server_reduce, ob_status_str, ob_unpack,
    OB_CONTROL_BYTES, OB_STATE_BLOCK, Tensors, adamw_hparams, control_create, control_fields, ob_adamw8_step,
    ob_adamw_hparams, ob_adamw_step, ob_grad_norm, ob_matmul, ob_product,
    MuonPlan, OB_MUON_MATCH_RMS, OB_MUON_PLAIN, OB_MUON_SHAPE, OB_NORM_2, OB_NORM_MAX, muon_hparams, ob_clip_grads,
    ob_muon_create, ob_muon_hparams, ob_muon_step, ob_tensor_norms, ob_tensor_norms_workspace,
    ob_state8_decode, ob_state8_encode, ob_tensors_create,
)
from .adamw import AdamW  # noqa: F401
from .muon import GradClip, Muon  # noqa: F401
from .schedule import OneBitAdam, OneBitLamb, step_kind  # noqa: F401
