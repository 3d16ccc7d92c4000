"""AdamW over a list of tensors: the states, the plan and the calls of
mx_grad_norm and mx_adamw, kept together (include/libmxmoe_train.h for the
arithmetic).  Nothing is read back by step(): it can be captured in a graph.
"""
import torch

from .training import BLOCK, mx_adamw, mx_adamw_plan, mx_grad_norm


class AdamW:
    """weights: float32 or bf16 GPU tensors (parameters too), updated in place
    by step(); grads: the tensors (float32 or bf16, same lengths) that hold
    their gradients at every step.  bf16 weights get float32 masters unless
    masters=False.  state_bits: 32, or 8 (E4M3 codes of m and sqrt(v) with a
    float32 scale per 256 elements, rounded at random without bias; the same
    step gives the same bits).  weight_decay: a number or one per tensor.
    max_norm: clip by the gradients' global norm; a step whose norm is
    infinite or NaN then changes nothing."""

    def __init__(self, weights, grads, lr=1e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.0, state_bits=32,
                 masters=True, max_norm=None):
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        if not weights:
            raise ValueError("no tensors")
        # (without autograd: the same memory, which step() writes through the plan)
        self.weights, self.grads = [w.detach() for w in weights], [g.detach() for g in grads]
        self.beta1, self.beta2 = betas
        self.eps, self.max_norm = eps, max_norm
        self.weight_decay = ([float(weight_decay)] * len(self.weights) if isinstance(weight_decay, (int, float))
                             else [float(d) for d in weight_decay])
        device = self.weights[0].device
        self.lr = torch.tensor([lr], dtype=torch.float32, device=device)
        self.steps = torch.zeros(2, dtype=torch.int64, device=device)
        self.norm = torch.zeros(2, dtype=torch.float32, device=device)
        self.masters = [w.float() if masters and w.dtype == torch.bfloat16 else None for w in self.weights]
        kind = torch.float32 if state_bits == 32 else torch.uint8

        def zeros(kind, length):
            return [torch.zeros(length(w), dtype=kind, device=device) for w in self.weights]

        self.m, self.v = (zeros(kind, lambda w: w.numel()) for _ in range(2))
        self.m_scale, self.v_scale = (
            (zeros(torch.float32, lambda w: -(-w.numel() // BLOCK)) for _ in range(2)) if state_bits == 8
            else (None, None))
        self.plan = mx_adamw_plan(self.weights, self.grads, self.m, self.v, masters=self.masters,
                                  m_scales=self.m_scale, v_scales=self.v_scale, weight_decay=self.weight_decay,
                                  unbiased=state_bits == 8)

    def set_lr(self, lr):
        self.lr.fill_(lr)

    def step(self):
        scale = None
        if self.max_norm is not None:
            scale = mx_grad_norm(self.plan, self.max_norm, out=self.norm)[1:]
        mx_adamw(self.plan, self.steps, lr=self.lr, beta1=self.beta1, beta2=self.beta2, eps=self.eps,
                 grad_scale=scale)

    def _tensors(self):
        lists = {"weights": self.weights, "masters": self.masters, "m": self.m, "v": self.v,
                 "m_scale": self.m_scale or [], "v_scale": self.v_scale or []}
        out = {f"{k}.{i}": t for k, ts in lists.items() for i, t in enumerate(ts) if t is not None}
        return {**out, "steps": self.steps, "lr": self.lr}

    def _settings(self):
        """What the constructor was given and a step depends on."""
        values = {"betas": [self.beta1, self.beta2], "eps": [self.eps], "weight_decay": self.weight_decay,
                  "max_norm": [-1.0 if self.max_norm is None else self.max_norm]}  # (-1: no clipping)
        return {k: torch.tensor(v, dtype=torch.float64) for k, v in values.items()}

    def state_dict(self):
        """Copies of everything that a later step depends on (weights and
        settings too)."""
        return {**{k: t.clone() for k, t in self._tensors().items()}, **self._settings()}

    def load_state_dict(self, state):
        """Into the tensors that are there: the plan stays valid.  The learning
        rate is loaded; other settings (betas, eps, weight decay, max_norm) are
        part of the plan and of captured steps, and have to be those of this
        optimizer (a state that has none of them is taken as it is)."""
        mine, settings = self._tensors(), self._settings()
        wanted = set(mine) | (set(settings) if set(settings) & set(state) else set())
        if set(state) != wanted or any(state[k].shape != t.shape or state[k].dtype != t.dtype
                                       for k, t in mine.items()):
            raise ValueError("the state is not of these tensors")
        for k, t in settings.items():
            if k in state and not torch.equal(state[k].double().cpu(), t):
                raise ValueError(f"{k}: the state was saved with {state[k].tolist()}, this optimizer has {t.tolist()}")
        for k, t in mine.items():
            t.copy_(state[k])
