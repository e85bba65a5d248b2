"""MultiAdam: the whole step of a list of tensors, one launch for the update of
all of them.

For parameters that were allocated one by one, or for the fragments of a ZeRO
rank's shard where tensors differ in their hyperparameters (norms and biases
without weight decay).  The step is ShardAdam's: the norm and overflow pass over
all gradients, the data-parallel exchange of its two scalars, the decision, the
update; host-scaled, or with the loss scaler and step counter in device memory
(device_state=True), where a step never waits and can be recorded in a torch
CUDA graph.  A recorded step keeps the hyperparameters (and the seed) that it was
recorded with, and reads the list's table: record it again to change them, and
keep the MultiAdam as long as the graph.
"""
from typing import Callable, Optional, Sequence

import torch

from . import AdamHyper, LossScaler, StepState, zero_adam_coef_bytes, zero_loss_scaler_update
from .moments8 import _codes_bytes, _scales_bytes, zero_moments8_pack
from .multi import (MAX_GROUPS, TensorTable, zero_multi_adam_step, zero_multi_adam_step_coef, zero_multi_decide_dev,
                    zero_multi_norm_decide_dev, zero_multi_norm_workspace_bytes, zero_multi_unscale_norm_overflow,
                    zero_multi_unscale_norm_overflow_dev)

_HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0)


def _slices(device, dtype, sizes):
    """One allocation cut into a zeroed tensor per entry of sizes, every tensor
    at a multiple of 256 bytes."""
    item = torch.empty(0, dtype=dtype).element_size()
    step = 256 // item
    at, starts = 0, []
    for k in sizes:
        starts.append(at)
        at += -(-k // step) * step
    flat = torch.zeros(at, dtype=dtype, device=device)
    return [flat[a:a + k] for a, k in zip(starts, sizes)]


class MultiAdam:
    def __init__(self, masters: Sequence[torch.Tensor], grads: Sequence[torch.Tensor],
                 params_out: Optional[Sequence[Optional[torch.Tensor]]] = None, *, hyper: Sequence[dict] = ({},),
                 groups: Optional[Sequence[int]] = None, max_grad_norm=0.0, state_bits: int = 32, moments=None,
                 scaler: Optional[LossScaler] = None, applied_steps: int = 0, device_state: bool = False,
                 tensor_norms: bool = False, seed: int = 0, device=None):
        """masters: fp32 tensors; grads: fp16, bf16 or fp32; params_out: the 16-bit
        copies (None entries: no copy).  hyper: one dict per group (lr, beta1,
        beta2, eps, weight_decay); groups: each tensor's group.  moments:
        (exp_avgs, exp_avg_sqs) fp32 lists to go on from, else zeros; with
        state_bits 8 they are rounded into the 8-bit format.  tensor_norms: the
        norm pass also fills self.tensor_sqnorm.  seed keys the rounding of 8-bit
        moments, with each tensor's and element's index: give each rank its own, else
        they round with the same words.  device: where an empty list keeps its scalars (its steps update
        nothing, but exchange and decide)."""
        if not len(grads) and device is None:
            raise ValueError("an empty list needs a device")
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits must be 32 or 8, got {state_bits}")
        if not 1 <= len(hyper) <= MAX_GROUPS:
            raise ValueError(f"1 to {MAX_GROUPS} groups expected, got {len(hyper)}")
        for h in hyper:
            if set(h) - set(_HYPER):
                raise ValueError(f"unknown hyperparameters {sorted(set(h) - set(_HYPER))}")
        self.hyper = [dict(_HYPER, **h, max_grad_norm=max_grad_norm) for h in hyper]
        if groups is not None and any(not 0 <= g < len(self.hyper) for g in groups):
            raise ValueError(f"groups must lie in [0, {len(self.hyper)})")
        self.groups = [0] * len(grads) if groups is None else [int(g) for g in groups]
        dev, sizes = grads[0].device if len(grads) else torch.device(device), [g.numel() for g in grads]
        if state_bits == 8:
            a = _slices(dev, torch.uint8, [_codes_bytes(n) for n in sizes])
            b = _slices(dev, torch.uint8, [_scales_bytes(n) for n in sizes])
        else:
            a, b = (_slices(dev, torch.float32, sizes) for _ in range(2))
        if moments is not None:
            if any(len(x) != len(sizes) for x in moments):
                raise ValueError("moments must hold one tensor per tensor of the list")
            for i, (m, v) in enumerate(zip(*moments)):
                if m.numel() != sizes[i] or v.numel() != sizes[i]:
                    raise ValueError(f"moments of tensor {i} differ from it in length")
                if state_bits == 8:
                    zero_moments8_pack(a[i], b[i], m, v)
                else:
                    a[i].copy_(m.reshape(-1))
                    b[i].copy_(v.reshape(-1))
        self.table = TensorTable(masters, a, b, grads, params_out, groups=self.groups, state_bits=state_bits)
        self.masters, self.exp_avgs, self.exp_avg_sqs = list(masters), a, b
        self.scaler = scaler if scaler is not None else LossScaler.static(1.0)
        self.t, self.seed = applied_steps, int(seed)
        self.workspace = torch.empty(zero_multi_norm_workspace_bytes(self.table), dtype=torch.uint8, device=dev)
        self.sqnorm = torch.empty(1, dtype=torch.float64, device=dev)
        self.overflow = torch.empty(1, dtype=torch.int32, device=dev)
        self.tensor_sqnorm = torch.empty(len(sizes), dtype=torch.float64, device=dev) if tensor_norms else None
        self._flag_host = torch.empty(1, dtype=torch.int32, pin_memory=True)
        self._flag_ready = torch.cuda.Event()
        self.state = StepState(self.scaler, applied_steps, dev) if device_state else None
        self.d_coefs = None
        if device_state:
            self.d_coefs = torch.empty(len(self.hyper) * zero_adam_coef_bytes(), dtype=torch.uint8, device=dev)
        self._graph = self._graph_key = None           # set when a checkpoint is loaded

    @classmethod
    def from_shard(cls, fragments, master: torch.Tensor, grad: torch.Tensor, param_out: Optional[torch.Tensor] = None, *,
                   groups: Sequence[int], moments=None, **kw) -> "MultiAdam":
        """The fragments of a rank's shard (zero_rank_fragments) as a list:
        views of the shard's flat buffers.  groups: the group of each of the
        model's tensors; moments: the shard's flat fp32 moments to go on from.
        The shard's padding is not touched; a rank that holds nothing else has an
        empty list, with which it takes part in the exchange and the decision.
        Where grad is an accumulated fp32 copy, which is already unscaled, steps
        need unscaled=True."""
        def cut(flat):
            return [flat[b:b + n] for _, _, b, n in fragments]
        kw.setdefault("device", master.device)
        return cls(cut(master), cut(grad), None if param_out is None else cut(param_out),
                   groups=[groups[t] for t, _, _, _ in fragments],
                   moments=None if moments is None else tuple(cut(m) for m in moments), **kw)

    def checkpoint_arrays(self) -> dict:
        names = ("master", "exp_avg", "exp_avg_sq") if self.table.state_bits == 32 else ("master", "moments8", "scales8")
        return {f"{name}_{i}": x for name, col in zip(names, (self.masters, self.exp_avgs, self.exp_avg_sqs))
                for i, x in enumerate(col)}

    def _hypers(self, **kw):
        return [AdamHyper(**h, **kw) for h in self.hyper]

    def step(self, grads: Optional[Sequence[torch.Tensor]] = None,
             allreduce: Optional[Callable[[torch.Tensor, torch.Tensor], None]] = None,
             unscaled: bool = False) -> Optional[bool]:
        """One full step.  grads: this step's gradients, where they are not in the
        buffers given before (the table is then built anew, which costs the host
        about a microsecond a tensor, and 0.07 ms per 1e9 elements); the list holds
        them until it is given others or release_grads() is called.  allreduce as in ShardAdam.step.
        unscaled: the gradients are already divided by the loss scale, as the fp32
        copy of ShardAdam.accumulate and reduce is: unlike ShardAdam, a list does
        not tell that from their type.  Returns True if the step was skipped (None
        with device_state)."""
        if grads is not None:
            self.table.set_grads(grads)
        if self.state is not None:
            if allreduce is None:
                zero_multi_norm_decide_dev(self.table, self._hypers(), self.state, self.sqnorm, self.overflow,
                                           self.d_coefs, self.workspace, self.tensor_sqnorm, unscaled)
            else:
                zero_multi_unscale_norm_overflow_dev(self.table, self.state, self.sqnorm, self.overflow, self.workspace,
                                                     self.tensor_sqnorm, unscaled)
                allreduce(self.sqnorm, self.overflow)
                zero_multi_decide_dev(self._hypers(), self.state, self.overflow, self.d_coefs, unscaled)
            zero_multi_adam_step_coef(self.table, self.d_coefs, len(self.hyper), self.sqnorm, self.overflow,
                                      self.state.applied(), seed=self.seed)
            return None
        inv = 1.0 if unscaled else 1.0 / self.scaler.scale
        zero_multi_unscale_norm_overflow(self.table, inv, self.sqnorm, self.overflow, self.workspace, self.tensor_sqnorm)
        if allreduce is not None:
            allreduce(self.sqnorm, self.overflow)
        zero_multi_adam_step(self.table, self._hypers(step=self.t + 1, inv_loss_scale=inv), self.sqnorm, self.overflow,
                             seed=self.seed)
        self._flag_host.copy_(self.overflow, non_blocking=True)
        self._flag_ready.record()
        self._flag_ready.synchronize()
        skip = zero_loss_scaler_update(self.scaler, bool(self._flag_host.item()))
        if not skip:
            self.t += 1
        return skip

    def release_grads(self) -> None:
        """After step(): let go of its gradients, so that clearing them (p.grad =
        None) frees their memory for the next backward pass.  The next step then
        has to be given its gradients."""
        self.table.release_grads()

    def read_state(self):
        """device_state: copy the state to the host (waits for the steps enqueued
        so far), refresh self.t and self.scaler from it and return it."""
        st = self.state.read()
        self.t = st.applied
        self.scaler.s = type(self.scaler.s).from_buffer_copy(bytes(st.scaler))
        return st
