"""AdamW for the layers of this package: one kernel launch a step for all of their tensors.

artiverse.ca "NVIDIA's 4-bit floating point pushes AI training limits" (paragraph on which parts
run in 4-bit): optimizer states and master weights stay in higher precision. The class only holds the
buffers and orders the calls; the arithmetic is nvfp4_adamw's.
"""
from __future__ import annotations

import torch

from . import AdamWPlan, AdamWTensor, NVFP4Error, adamw
from .linear import NVFP4Linear, _state_of


class AdamW:
    """entries: (parameter, gradient, weight_decay) triples, or (parameter, gradient) with the default
    decay. A BF16 parameter gets an FP32 master copy, which follows it where it is changed between steps
    (as far as torch counts changes: not through .data); an FP32 one is updated itself. The gradient
    (FP32 or BF16, the parameter's shape) is read where it is at every step.

    states: "fp32", or "8bit" (two bytes and a sixteenth per element instead of eight).
    max_norm: clip the gradients' norm over all tensors; step() then returns the norm (a device
    float [1]), and a step whose norm is not finite changes nothing but the step count.
    amax: device float, one per tensor: max|weight| after the latest step.
    """

    def __init__(self, entries, lr: float = 3e-4, betas=(0.9, 0.95), eps: float = 1e-8, weight_decay: float = 0.1,
                 states: str = "fp32", max_norm: float | None = None, seed: int = 0, layers=()):
        if states not in ("fp32", "8bit"):
            raise NVFP4Error(f"unknown states {states!r}: fp32 or 8bit")
        self.lr, self.betas, self.eps, self.max_norm, self.seed = lr, betas, eps, max_norm, seed
        self.states, self.steps = states, 0
        self.params, self.grads, self.masters, tensors = [], [], [], []
        self._sources = []                                   # (parameter as given, its address)
        self._places = []                                    # (a layer's parameters, name, its address)
        self._held = []                                      # (owner of a gradient, attribute, its address)
        named = set()
        for entry in entries:
            param, grad, *decay = entry
            p = param.detach()
            if p.dtype not in (torch.bfloat16, torch.float32) or not p.is_contiguous():
                raise NVFP4Error("parameters must be contiguous bfloat16 or float32 tensors")
            if grad is None or grad.shape != p.shape:
                raise NVFP4Error("every parameter needs a gradient of its shape that stays where it is")
            if p.numel() and p.data_ptr() in named:
                raise NVFP4Error("a parameter is named twice: give it one entry, with the sum of its gradients")
            named.add(p.data_ptr())
            master = p.float() if p.dtype == torch.bfloat16 else p
            tensors.append(AdamWTensor(p=master, grad=grad, weight_decay=decay[0] if decay else weight_decay,
                                       w_out=p if p.dtype == torch.bfloat16 else None, **self._state(p)))
            self.params.append(p)
            self.grads.append(grad)
            self._sources.append((param, p.data_ptr()))
            if param.is_leaf and param.grad is grad:
                self._held.append((param, "grad", grad.data_ptr()))
            self.masters.append(master)
        self.plan = AdamWPlan(tensors)
        self.amax = torch.zeros((len(tensors),), dtype=torch.float32, device=self.plan.device)
        self._layers = list(layers)                          # (index of the weight, layer)
        self._amaxes = [(self.amax[i:i + 1], self.params[i], layer) for i, layer in self._layers]
        self._mains = []                                     # (parameter, its main gradient)
        self._counted = [p for p in self.params if not p.is_inference()]     # torch counts their changes
        self._followed = [(p, m) for p, m in zip(self.params, self.masters) if p is not m and not p.is_inference()]
        self._see()

    def _see(self):
        self._seen = [p._version for p, _ in self._followed]

    def _follow_parameters(self):
        """Masters of parameters that changed since the last step: where the BF16 value is no longer the
        master's, the parameter's."""
        for (p, m), seen in zip(self._followed, self._seen):
            if p._version != seen:
                m.copy_(torch.where(p == m.bfloat16(), m, p.float()))
        self._see()

    def _state(self, p):
        n, dev = p.numel(), p.device
        if self.states == "fp32":
            return {k: torch.zeros((n,), dtype=torch.float32, device=dev) for k in ("m", "v")}
        return {k: torch.zeros((n if len(k) == 1 else (n + 31) // 32,), dtype=torch.uint8, device=dev)
                for k in ("m", "v", "m_scale", "v_scale")}

    @classmethod
    def of(cls, module: torch.nn.Module, weight_decay: float = 0.1, **kw):
        """Of every parameter of a module that requires a gradient now: NVFP4Linear weights with their
        main_grad and decay, their biases and every other parameter of one dimension without decay. A
        parameter without a main gradient gets a .grad that has to stay in place (zero_grad of this
        class, not set_to_none). A parameter that several layers share is stepped once, with all of
        their gradients: the layers share one main gradient from here on, and what other uses of the
        parameter leave in its .grad is added there by step()."""
        entries, layers, held, places, at = [], [], [], [], {}
        for m in module.modules():
            if not isinstance(m, NVFP4Linear):
                continue
            for name, main, decay in (("weight", "main_grad", weight_decay), ("bias", "bias_main_grad", 0.0)):
                p, grad = getattr(m, name), getattr(m, main)
                if grad is None or not p.requires_grad:
                    continue
                if id(p) not in at:
                    at[id(p)] = len(entries)
                    entries.append((p, grad, decay))
                elif grad is not entries[at[id(p)]][1]:
                    entries[at[id(p)]][1].add_(grad)
                    setattr(m, main, entries[at[id(p)]][1])
                places.append((m._parameters, name, p.data_ptr()))
                held.append((m, main, entries[at[id(p)]][1].data_ptr()))
                if name == "weight":
                    layers.append((at[id(p)], m))
        mains = [(p, grad) for p, grad, _ in entries]
        for p in module.parameters():
            if id(p) in at or not p.requires_grad:
                continue
            if p.grad is None:
                p.grad = torch.zeros_like(p)
            entries.append((p, p.grad, weight_decay if p.dim() > 1 else 0.0))
        opt = cls(entries, weight_decay=weight_decay, layers=layers, **kw)
        opt._mains = mains
        opt._held += held
        opt._places += places
        return opt

    def step(self, lr: float | None = None):
        """One step; returns the gradients' norm with max_norm, else None. The kernel reads and writes
        the buffers that the optimizer was made with: one that has been replaced since is an error."""
        for param, address in self._sources:
            if param.data_ptr() != address:
                self._moved("data of a parameter")
        for parameters, name, address in self._places:
            now = parameters.get(name)
            if now is None or now.data_ptr() != address:
                self._moved(f"{name} of a layer")
        for owner, name, address in self._held:
            now = getattr(owner, name)
            if now is None or now.data_ptr() != address:
                self._moved(f"{name} of a {type(owner).__name__}")
        for p, main in self._mains:
            if p.grad is not None:                           # of a use without the main gradient
                main.add_(p.grad)
                p.grad = None
        self._follow_parameters()
        norm = adamw(self.plan, lr=self.lr if lr is None else lr, betas=self.betas, eps=self.eps, step=self.steps + 1,
                     max_norm=self.max_norm, seed=self.seed, amax_out=self.amax)
        self.steps += 1
        # the kernel wrote them: autograd and the layers are to see it
        torch.autograd.graph.increment_version(self._counted)
        self._see()
        for amax, param, layer in self._amaxes:
            layer.__dict__["_weight_amax"] = amax, _state_of(param)       # layer.weight_amax, without Module's ways
        return norm

    @staticmethod
    def _moved(what):
        raise NVFP4Error(f"the {what} has moved since the optimizer was made: clear gradients with its zero_grad, and make "
                         f"it anew after moving parameters")

    def zero_grad(self):
        torch._foreach_zero_(self.grads)
        for p, _ in self._mains:
            p.grad = None

    def state_dict(self) -> dict:
        self._follow_parameters()
        keys = ("m", "v") if self.states == "fp32" else ("m", "v", "m_scale", "v_scale")
        return {"states": self.states, "steps": self.steps, "seed": self.seed,
                "masters": [m.clone() for m in self.masters],
                **{k: [getattr(t, k).clone() for t in self.plan.tensors] for k in keys}}

    def load_state_dict(self, state: dict):
        """Restores masters, states and step count, and the BF16 weights from the masters."""
        keys = ("m", "v") if self.states == "fp32" else ("m", "v", "m_scale", "v_scale")
        pairs = [(self.masters, state["masters"])] if state["states"] == self.states else []
        pairs += [([getattr(t, k) for t in self.plan.tensors], state[k]) for k in keys if pairs]
        if not pairs or any([a.shape for a in mine] != [b.shape for b in theirs] for mine, theirs in pairs):
            raise NVFP4Error("the state is of another optimizer")
        for mine, theirs in pairs:
            for a, b in zip(mine, theirs):
                a.copy_(b)
        for p, m in zip(self.params, self.masters):
            if p is not m:
                p.copy_(m)
        self._see()
        for _, layer in self._layers:
            layer.weight_amax = None                         # of the weights before
        self.steps, self.seed = state["steps"], state["seed"]
