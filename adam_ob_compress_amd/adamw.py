"""AdamW over a model's parameter tensors, a driver over ob_grad_norm, ob_adamw_step and ob_adamw8_step (no
arithmetic here).

It stands beside OneBitAdam: OneBitAdam steps one flat fp32 buffer and compresses what workers exchange;
AdamW steps the tensors of a model where they lie, in their own types.  Their state layouts differ (one flat
buffer; each tensor's part from a multiple of 256 elements), and nothing converts one into the other.
"""
from __future__ import annotations

import torch

from . import _native as nat

_ROUNDING = {"nearest": nat.OB_ROUND_NEAREST, "stochastic": nat.OB_ROUND_STOCHASTIC}


class ListOptimizer:
    """What the optimizers over a model's tensors share: their parameters, the list that describes them, the control block and
    a master copy."""

    def _collect(self, params, lr, weight_decay, common):
        """Parameters and their factors of rate and decay from tensors or groups; common: what no group may have of its own."""
        if isinstance(params, torch.Tensor):
            raise TypeError("params must be a list of tensors or groups, got a tensor")
        groups = list(params)
        if groups and not isinstance(groups[0], dict):
            groups = [{"params": groups}]
        self.params, lr_mults, wd_mults = [], [], []
        for group in groups:
            for k, own in common.items():
                if k in group and (group[k] if k != "betas" else tuple(group[k])) != own:
                    raise ValueError(f"a group cannot have its own {k}")
            for p in [group["params"]] if isinstance(group["params"], torch.Tensor) else group["params"]:
                self.params.append(p)
                lr_mults.append(_ratio(group.get("lr", lr), lr, "lr"))
                wd_mults.append(_ratio(group.get("weight_decay", weight_decay), weight_decay, "weight_decay"))
        if not self.params:
            raise ValueError("no parameters")
        if len({id(p) for p in self.params}) < len(self.params):
            raise ValueError("a parameter is listed twice")
        dev = self.params[0].device
        for j, p in enumerate(self.params):
            if p.device != dev:
                raise ValueError(f"all parameters must be on {dev} (got {p.device})")
            if not p.is_contiguous():
                raise ValueError(f"parameter {j} must be contiguous")
        self._no_leaves = [(j, p) for j, p in enumerate(self.params) if not p.is_leaf]
        return lr_mults, wd_mults

    def _begin(self, lr_mults, wd_mults, grad_dtype, master, max_norm):
        """The list, the master copy and the control block."""
        dev = self.params[0].device
        self.max_norm = max_norm
        self.list = nat.ob_tensors_create([p.numel() for p in self.params],
                                          grad_dtype or [p.dtype for p in self.params],
                                          [p.dtype for p in self.params], lr_mults, wd_mults, dev)
        self._index = self.list.device.index
        self.master = None
        if master:
            self.master = torch.zeros(self.list.state_elems, dtype=torch.float32, device=dev)
            for t, p in enumerate(self.params):
                self._part(self.master, t).copy_(p.detach())
        self.control = nat.control_create(dev) if max_norm is not None else None

    def _gradients(self, grads):
        if grads is not None:
            return list(grads)
        for j, p in self._no_leaves:
            if not p.retains_grad and p.grad is None:   # its .grad stays None, as of a parameter to leave alone
                raise ValueError(f"parameter {j} is no leaf and has no .grad of its own: give the gradients to step")
        return [p.grad for p in self.params]

    def _part(self, flat, t):
        """Tensor t's part of a flat state buffer, in the parameter's shape."""
        o, p = self.list.state_offset(t), self.params[t]
        return flat[o:o + p.numel()].view(p.shape)

    def _capturing(self, stream):
        """Whether the stream that a step is enqueued on is being captured."""
        if stream is None:
            if torch._C._cuda_getDevice() == self._index:   # what current_device() asks
                return torch.cuda.is_current_stream_capturing()
            stream = torch.cuda.current_stream(self.list.device)
        elif not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), self.list.device)
        with torch.cuda.stream(stream):
            return torch.cuda.is_current_stream_capturing()

    def set_lr_scale(self, factor: float):
        """Factor of every rate from the next step or replay on (needs max_norm)."""
        if self.control is None:
            raise ValueError("a factor of the rate needs max_norm (inf: no clipping); without it change hp.lr")
        nat.control_fields(self.control)["lr_scale"].fill_(factor)

    @property
    def norm(self):
        """The last step's gradient norm before clipping, on the GPU (None without max_norm)."""
        return None if self.control is None else nat.control_fields(self.control)["norm"]

    def steps(self) -> int:
        """Steps taken (waits for the GPU with max_norm)."""
        return self.hp.step if self.control is None else int(nat.control_fields(self.control)["step"])


class AdamW(ListOptimizer):
    """AdamW with decoupled weight decay, states in fp32 or in 8 bits.

    ``params``: tensors (fp32, bf16, fp16; contiguous, on one GPU), or parameter groups as dicts with "params" (tensors, or
    one) and optionally "lr" and "weight_decay", which can not be changed later on; no other argument can differ between
    groups, and a common value of 0 allows no other.  ``state_bits``: 32 or 8.  ``master``: keep fp32 master copies of 16-bit
    parameters (taken from them here).  ``max_norm``: clip by the global gradient norm and leave out steps whose norm is
    not finite (inf, 0 or less: only the latter); None: neither.  ``rounding="stochastic"`` rounds 8-bit states and
    16-bit parameters without a master by chance, with bits from (``sr_seed``, the step).

    ``step()`` takes ``p.grad`` of every parameter (or the list it is given); a parameter without a gradient is
    left alone.  Everything is enqueued on the current stream and nothing waits for the GPU, so a step can be captured
    into a HIP graph; with ``max_norm`` the step count then lives in ``self.control``, where a replay
    advances it, and ``set_lr_scale`` changes the rate between replays; the optimizer must outlive the graph.  Without
    ``max_norm`` the count is a host value, which a captured step would repeat: capturing then raises.

    ``self.hp`` holds the step's parameters; what is changed there (``hp.lr``) holds from the next step on.  The groups'
    rates and decays keep their ratios to it.
    """

    def __init__(self, params, *, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, max_norm=None,
                 state_bits=32, master=False, rounding="nearest", sr_seed=0, bias_correction=True, grad_dtype=None):
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits must be 8 or 32, got {state_bits}")
        common = dict(betas=tuple(betas), eps=eps, max_norm=max_norm, state_bits=state_bits, master=master, rounding=rounding,
                      sr_seed=sr_seed, bias_correction=bias_correction, grad_dtype=grad_dtype, amsgrad=False, maximize=False)
        self.state_bits = state_bits
        self._begin(*self._collect(params, lr, weight_decay, common), grad_dtype, master, max_norm)
        self.hp = nat.adamw_hparams(lr=lr, beta1=betas[0], beta2=betas[1], eps=eps, weight_decay=weight_decay,
                                    bias_correction=bias_correction, step=0, rounding=_ROUNDING[rounding], sr_seed=sr_seed)
        N, dev = self.list.state_elems, self.params[0].device
        self.m = self.v = self.m_codes = self.m_scales = self.v_codes = self.v_scales = None
        if state_bits == 32:
            self.m, self.v = (torch.zeros(N, dtype=torch.float32, device=dev) for _ in range(2))
        else:
            self.m_codes = torch.zeros(N, dtype=torch.int8, device=dev)
            self.v_codes = torch.zeros(N, dtype=torch.uint8, device=dev)
            self.m_scales, self.v_scales = (torch.zeros(N // nat.OB_STATE_BLOCK, dtype=torch.float32, device=dev)
                                            for _ in range(2))

    @torch.no_grad()
    def step(self, grads=None, loss_scale: float = 1.0, stream=None):
        """One step; loss_scale: what the gradients were multiplied with (other than 1 needs max_norm)."""
        grads = self._gradients(grads)
        norm = None
        if self.control is not None:
            norm = (1.0 / loss_scale, self.max_norm)
        else:
            if loss_scale != 1.0:
                raise ValueError("a loss scale needs max_norm (inf: no clipping)")
            if self._capturing(stream):
                raise RuntimeError("a captured step needs max_norm (inf: no clipping): its count is kept on the GPU")
            self.hp.step += 1
        try:
            if self.state_bits == 32:
                nat.ob_adamw_step(self.list, grads, self.params, self.m, self.v, self.hp, self.master, self.control, stream,
                                  norm)
            else:
                nat.ob_adamw8_step(self.list, grads, self.params, self.m_codes, self.m_scales, self.v_codes,
                                   self.v_scales, self.hp, self.master, self.control, stream, norm)
        except Exception:
            if self.control is None:
                self.hp.step -= 1   # a refused step is not counted
            raise

    def moments(self):
        """The flat moments (m, v) in fp32; with 8-bit states what the codes stand for, in new tensors."""
        if self.state_bits == 32:
            return self.m, self.v
        m = torch.empty(self.list.state_elems, dtype=torch.float32, device=self.m_codes.device)
        v = torch.empty_like(m)
        nat.ob_state8_decode(self.m_codes, self.m_scales, self.v_codes, self.v_scales, m, v)
        return m, v

    _STATES = ("m", "v", "m_codes", "m_scales", "v_codes", "v_scales", "master")

    def state_dict(self) -> dict:
        """Step count and flat states (references), with max_norm also the factor of set_lr_scale and the count of steps
        left out.  Restored into an AdamW made with the same arguments, with the same values in hp, it gives
        the same steps bit for bit."""
        d = {"step": self.steps(), "state_bits": self.state_bits,
             **{k: getattr(self, k) for k in self._STATES if getattr(self, k) is not None}}
        if self.control is not None:
            f = nat.control_fields(self.control)
            d.update(lr_scale=float(f["lr_scale"]), skipped=int(f["skipped"]))
        return d

    def load_state_dict(self, d: dict):
        """Restore a state_dict of the same list, also one with states of the other width.  What it does not hold of
        the rate's factor and the steps left out stays as it is."""
        if (self.master is None) != ("master" not in d):
            raise ValueError("the state has a master copy and this optimizer none, or the other way round")
        if self.control is None and d.get("lr_scale", 1.0) != 1.0:
            raise ValueError("the state has a factor of the rate (lr_scale), which needs max_norm")
        if d.get("state_bits") not in (8, 32):
            raise ValueError(f"state_bits must be 8 or 32, got {d.get('state_bits')}")
        if not isinstance(d.get("step"), int):
            raise ValueError(f"step must be a whole number, got {d.get('step')}")
        dev = self.list.device
        for k in self._STATES[:2] if d["state_bits"] == 32 else self._STATES[2:6]:
            if not isinstance(d.get(k), torch.Tensor):
                raise ValueError(f"the state lacks {k}")
        for k in self._STATES:
            want = self.list.state_elems // (nat.OB_STATE_BLOCK if k.endswith("_scales") else 1)
            if k in d and d[k].numel() != want:
                raise ValueError(f"{k} must have {want} elements, got {d[k].numel()}")
        d = {k: x.to(dev).reshape(-1) if k in self._STATES else x for k, x in d.items()}
        if d["state_bits"] == self.state_bits:
            for k in self._STATES[:2] if self.state_bits == 32 else self._STATES[2:6]:
                getattr(self, k).copy_(d[k])
        elif self.state_bits == 8:
            nat.ob_state8_encode(d["m"], d["v"], self.m_codes, self.m_scales, self.v_codes, self.v_scales)
        else:
            nat.ob_state8_decode(d["m_codes"], d["m_scales"], d["v_codes"], d["v_scales"], self.m, self.v)
        if self.master is not None:
            self.master.copy_(d["master"])
        self.hp.step = d["step"]
        if self.control is not None:
            f = nat.control_fields(self.control)
            for k in ("step", "lr_scale", "skipped"):
                if k in d:
                    f[k].fill_(d[k])


def _ratio(value, base, name):
    """A group's value as a factor of the common one."""
    if value == base:
        return 1.0
    if base == 0:
        raise ValueError(f"a group has its own {name}, so the common {name} must not be 0")
    return value / base
