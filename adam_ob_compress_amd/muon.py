"""Muon over a model's matrices, and clipping over what several optimizers step: drivers over ob_muon_step, ob_tensor_norms and
ob_clip_grads (no arithmetic here)."""
from __future__ import annotations

import torch

from . import _native as nat
from .adamw import ListOptimizer

_SCALE = {"plain": nat.OB_MUON_PLAIN, "shape": nat.OB_MUON_SHAPE, "match_rms": nat.OB_MUON_MATCH_RMS}
_NORM = {"2": nat.OB_NORM_2, "max": nat.OB_NORM_MAX}


class Muon(ListOptimizer):
    """Muon: momentum, orthogonalised by five polynomial iterations, with decoupled weight decay; for a model's matrices, beside
    AdamW for its vectors and embeddings.

    ``params``: tensors of two dimensions, or of more for matrices behind each other (experts, heads): the last two are rows and
    columns.  fp32, bf16 or fp16, contiguous, on one GPU; or parameter groups, as in AdamW.  ``scale``: what the orthogonal
    matrix is multiplied with: "match_rms" 0.2 sqrt(max(rows, columns)), so that AdamW's rates and decays fit, "shape"
    sqrt(max(1, rows / columns)), "plain" 1.  ``master``, ``max_norm``, ``step()``, ``set_lr_scale``, ``hp`` as in AdamW; 16-bit
    parameters are rounded to nearest.

    ``max_norm`` clips by the norm over this optimizer's gradients and keeps the step count on the GPU.  Without it a step may be
    captured too, and the count is of the calls of ``step()``.  Gradients that AdamW steps as well belong to one norm: give
    them all to GradClip first, and ``max_norm=inf`` to both optimizers if steps whose norm is not finite shall be left out.

    The workspace (4 bytes per element and 4 r^2 per matrix, r the smaller side, so 8 bytes per element of a square one, for the matrices that
    go through the iterations together: at most about 2 GB for a list of many) is kept with the optimizer, so its steps must not
    overlap each other.
    """

    def __init__(self, params, *, lr=1e-3, momentum=0.95, weight_decay=0.1, max_norm=None, nesterov=True, iterations=5, eps=1e-7,
                 scale="match_rms", master=False, grad_dtype=None):
        if scale not in _SCALE:
            raise ValueError(f"scale must be one of {', '.join(_SCALE)}, got {scale}")
        common = dict(momentum=momentum, max_norm=max_norm, nesterov=nesterov, iterations=iterations, eps=eps, scale=scale,
                      master=master, grad_dtype=grad_dtype)
        mults = self._collect(params, lr, weight_decay, common)
        for j, p in enumerate(self.params):
            if p.dim() < 2:
                raise ValueError(f"parameter {j} is no matrix (shape {tuple(p.shape)}): AdamW steps it")
        self._begin(*mults, grad_dtype, master, max_norm)
        dev = self.params[0].device
        self.hp = nat.muon_hparams(lr=lr, momentum=momentum, weight_decay=weight_decay, eps=eps, nesterov=nesterov,
                                   iterations=iterations, scale=_SCALE[scale])
        self.plan = nat.ob_muon_create(self.list, [p.shape for p in self.params])
        self.m = torch.zeros(self.list.state_elems, dtype=torch.float32, device=dev)
        self.workspace = torch.empty(self.plan.workspace_bytes, dtype=torch.uint8, device=dev)
        self._calls = 0

    def steps(self) -> int:
        """Steps taken (waits for the GPU with max_norm)."""
        return self._calls if self.control is None else int(nat.control_fields(self.control)["step"])

    @torch.no_grad()
    def step(self, grads=None, loss_scale: float = 1.0, stream=None):
        """One step; loss_scale: what the gradients were multiplied with (other than 1 needs max_norm)."""
        grads = self._gradients(grads)
        norm = None
        if self.control is not None:
            norm = (1.0 / loss_scale, self.max_norm)
        elif loss_scale != 1.0:
            raise ValueError("a loss scale needs max_norm (inf: no clipping)")
        nat.ob_muon_step(self.plan, grads, self.params, self.m, self.hp, self.workspace, self.master, self.control, stream, norm)
        self._calls += 1

    def state_dict(self) -> dict:
        """Step count and flat states (references), with max_norm also the factor of set_lr_scale and the count of steps
        left out.  Restored into a Muon made with the same arguments, with the same values in hp, it gives the same steps
        bit for bit."""
        d = {"step": self.steps(), "m": self.m}
        if self.master is not None:
            d["master"] = self.master
        if self.control is not None:
            f = nat.control_fields(self.control)
            d.update(lr_scale=float(f["lr_scale"]), skipped=int(f["skipped"]))
        return d

    def load_state_dict(self, d: dict):
        """Restore a state_dict of the same list.  What it does not hold of the rate's factor and the steps left out stays as
        it is."""
        if (self.master is None) != ("master" not in d):
            raise ValueError("the state has a master copy and this optimizer none, or the other way round")
        if self.control is None and d.get("lr_scale", 1.0) != 1.0:
            raise ValueError("the state has a factor of the rate (lr_scale), which needs max_norm")
        if not isinstance(d.get("step"), int):
            raise ValueError(f"step must be a whole number, got {d.get('step')}")
        names = ["m"] + (["master"] if self.master is not None else [])
        for k in names:
            if not isinstance(d.get(k), torch.Tensor):
                raise ValueError(f"the state lacks {k}")
            if d[k].numel() != self.list.state_elems:
                raise ValueError(f"{k} must have {self.list.state_elems} elements, got {d[k].numel()}")
        for k in names:
            getattr(self, k).copy_(d[k].reshape(-1))
        self._calls = d["step"]
        if self.control is not None:
            f = nat.control_fields(self.control)
            for k in ("step", "lr_scale", "skipped"):
                if k in d:
                    f[k].fill_(d[k])


class GradClip:
    """Clips the gradients of many tensors in place, by the norm of all or (``per_tensor``) each by its own; for gradients that
    more than one optimizer steps.

    The workspace and the norms are kept with it, so its calls must not overlap each other.  The norm is over the gradients
    given, on this GPU.  Where workers hold parts of them (sharded gradients), ob_tensor_norms and ob_clip_grads are called in its
    place, with the norms joined over the workers between the two.

    ``params``: the tensors whose ``.grad`` is clipped (contiguous, on one GPU), each once.  ``norm``: "2" or "max".  Everything
    is enqueued on the current stream and nothing waits for the GPU, so a call can be captured.  A norm that is not finite makes
    the gradients NaN, so that optimizers with ``max_norm=inf`` leave the step out.
    """

    def __init__(self, params, *, max_norm, norm="2", per_tensor=False, grad_dtype=None):
        if norm not in _NORM:
            raise ValueError(f"norm must be one of {', '.join(_NORM)}, got {norm}")
        if isinstance(params, torch.Tensor):
            raise TypeError("params must be a list of tensors, got a tensor")
        self.params = list(params)
        if not self.params:
            raise ValueError("no parameters")
        if len({id(p) for p in self.params}) < len(self.params):
            raise ValueError("a parameter is listed twice")
        dev = self.params[0].device
        for p in self.params:
            if p.device != dev:
                raise ValueError(f"all parameters must be on {dev} (got {p.device})")
        self.max_norm, self.kind, self.per_tensor = max_norm, _NORM[norm], per_tensor
        dtypes = grad_dtype or [p.dtype for p in self.params]
        self.list = nat.ob_tensors_create([p.numel() for p in self.params], dtypes, dtypes, device=dev)
        self.norms = torch.zeros(len(self.params) + 1, dtype=torch.float32, device=dev)
        self.workspace = torch.empty(self.list.norm_bytes, dtype=torch.uint8, device=dev)

    @torch.no_grad()
    def __call__(self, grads=None, loss_scale: float = 1.0, stream=None):
        """Clip ``.grad`` of every parameter (or the list given; None: no gradient), divided by loss_scale.  Returns the norm of
        all before clipping, one element on the GPU; each tensor's is in ``self.norms``."""
        grads = [p.grad for p in self.params] if grads is None else list(grads)
        nat.ob_tensor_norms(self.list, grads, self.norms, 1.0 / loss_scale, self.kind, self.workspace, stream)
        nat.ob_clip_grads(self.list, grads, self.norms, self.max_norm, 1.0 / loss_scale, None, self.per_tensor, stream)
        return self.norms[-1:]
