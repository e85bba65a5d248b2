"""MultiMuon: the whole step of a list of matrices by orthogonalised momentum.

For the hidden matrices of a model (embeddings, heads, norms and biases keep
AdamW: MultiAdam).  The step is MultiAdam's up to the update: the norm and
overflow pass over all gradients, the data-parallel exchange of its two scalars
and the decision; then the momentum pass, the orthogonalisation of its updates,
in their place, and the update of masters and copies.  Host-scaled, or with the
loss scaler and step counter in device memory (device_state=True), where a step
never waits and can be recorded in a torch CUDA graph; a recorded step keeps its
hyperparameters and reads the list's tables: record it again to change them, and
keep the MultiMuon as long as the graph.

An update needs its whole matrix.  Across data-parallel ranks, give each rank
whole matrices: a list of those whose fragment (zero_rank_fragments) holds all of
the matrix, or matrices gathered before the step.
"""
import math
from typing import Callable, Optional, Sequence

import torch

from . import AdamHyper, LossScaler, StepState, zero_adam_coef_bytes, zero_loss_scaler_update
from .matrices import (MatrixTable, MuonHyper, ORTHO_COEFS, zero_multi_momentum_step, zero_multi_momentum_step_coef,
                       zero_multi_muon_update, zero_multi_orthogonalize, zero_multi_orthogonalize_workspace_bytes)
from .multi import (MAX_GROUPS, TensorTable, zero_multi_decide_dev, zero_multi_norm_decide_dev,
                    zero_multi_norm_workspace_bytes, zero_multi_unscale_norm_overflow,
                    zero_multi_unscale_norm_overflow_dev)
from .multi_adam import _slices

_HYPER = dict(lr=2e-2, momentum=0.95, weight_decay=0.0, nesterov=True)


def muon_scale(shape: Sequence[int], adjust: Optional[str]) -> float:
    """The factor of the learning rate for a matrix of this shape.  An orthogonal
    rows x cols matrix has elements of root mean square 1 / sqrt(max(rows, cols)).
    "rms": 0.2 sqrt(max(rows, cols)), so that elements move about as AdamW's;
    "spectral": sqrt(max(1, rows / cols)); None: 1."""
    rows, cols = shape[-2:]
    if adjust is None or not rows or not cols:
        return 1.0
    if adjust == "rms":
        return 0.2 * math.sqrt(max(rows, cols))
    if adjust == "spectral":
        return math.sqrt(max(1.0, rows / cols))
    raise ValueError(f"adjust must be 'rms', 'spectral' or None, got {adjust!r}")


class MultiMuon:
    def __init__(self, masters: Sequence[torch.Tensor], grads: Sequence[torch.Tensor],
                 params_out: Optional[Sequence[Optional[torch.Tensor]]] = None, *, hyper: Sequence[dict] = ({},),
                 groups: Optional[Sequence[int]] = None, adjust: Optional[str] = "rms", max_grad_norm=0.0,
                 coefs=ORTHO_COEFS, eps: float = 1e-7, momentums=None, update_dtype=torch.bfloat16,
                 scaler: Optional[LossScaler] = None, applied_steps: int = 0, device_state: bool = False,
                 tensor_norms: bool = False, device=None):
        """masters: fp32 matrices, or batches of matrices in three dimensions;
        grads: fp16, bf16 or fp32; params_out: the 16-bit copies (None entries: no
        copy).  hyper: one dict per group (lr, momentum, weight_decay, nesterov);
        groups: each matrix's group.  adjust: how the learning rate goes by the
        shape (muon_scale).  coefs, eps: the orthogonalisation's.  momentums: fp32
        matrices to go on from, else zeros.  update_dtype: bf16, or fp16 where
        unscaled gradients keep clear of its ends.  tensor_norms: the norm pass
        also fills self.tensor_sqnorm.  device: where an empty list keeps its
        scalars."""
        if not len(grads) and device is None:
            raise ValueError("an empty list needs a device")
        if update_dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"update_dtype must be bfloat16 or float16, got {update_dtype}")
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
        shapes = [tuple(m.shape) for m in masters]
        if len(shapes) != len(sizes) or any(math.prod(x) != n for x, n in zip(shapes, sizes)):
            raise ValueError("masters and grads differ in their shapes")
        ms = [x.view(shape) for x, shape in zip(_slices(dev, torch.float32, sizes), shapes)]
        if momentums is not None:
            if len(momentums) != len(ms) or any(tuple(a.shape) != tuple(b.shape) for a, b in zip(momentums, ms)):
                raise ValueError("momentums must hold one matrix per matrix of the list, of its shape")
            for a, b in zip(ms, momentums):
                a.copy_(b)
        updates = [x.view(shape) for x, shape in zip(_slices(dev, update_dtype, sizes), shapes)]
        self.scales, self.update_dtype = [muon_scale(shape, adjust) for shape in shapes], update_dtype
        self.table = MatrixTable(updates, None, ms, list(grads), masters, params_out, scales=self.scales,
                                 groups=self.groups)
        self.norm_table = TensorTable.of_grads(grads)
        self.masters, self.momentums, self.updates = list(masters), ms, updates
        self.coefs, self.eps = tuple(tuple(float(c) for c in x) for x in coefs), float(eps)
        self.scaler = scaler if scaler is not None else LossScaler.static(1.0)
        self.t = applied_steps
        self.workspace = torch.empty(max(1, zero_multi_orthogonalize_workspace_bytes(self.table)), dtype=torch.uint8, device=dev)
        self.norm_workspace = torch.empty(zero_multi_norm_workspace_bytes(self.norm_table), dtype=torch.uint8, device=dev)
        self.sqnorm = torch.empty(1, dtype=torch.float64, device=dev)
        self.overflow = torch.empty(1, dtype=torch.int32, device=dev)
        self.tensor_sqnorm = torch.empty(len(sizes), dtype=torch.float64, device=dev) if tensor_norms else None
        self._flag_host = torch.empty(1, dtype=torch.int32, pin_memory=True)
        self._flag_ready = torch.cuda.Event()
        self.state = StepState(self.scaler, applied_steps, dev) if device_state else None
        self.d_coefs = torch.empty(zero_adam_coef_bytes(), dtype=torch.uint8, device=dev) if device_state else None
        self._graph = self._graph_key = None           # set when a checkpoint is loaded

    def checkpoint_arrays(self) -> dict:
        return {f"{name}_{i}": x for name, col in (("master", self.masters), ("momentum", self.momentums))
                for i, x in enumerate(col)}

    def checkpoint_settings(self) -> dict:
        """What a resumed list has to agree in, as JSON holds it."""
        return dict(coefs=[list(x) for x in self.coefs], eps=self.eps, scales=list(self.scales),
                    update_dtype=str(self.update_dtype).replace("torch.", ""))

    def _hypers(self):
        return [MuonHyper(**{k: v for k, v in h.items() if k != "max_grad_norm"}) for h in self.hyper]

    def step(self, grads: Optional[Sequence[torch.Tensor]] = None,
             allreduce: Optional[Callable[[torch.Tensor, torch.Tensor], None]] = None,
             unscaled: bool = False) -> Optional[bool]:
        """One full step.  grads: this step's gradients, where they are not in the
        buffers given before; the list holds them until it is given others or
        release_grads() is called.  allreduce as in ShardAdam.step.  unscaled: the
        gradients are already divided by the loss scale.  Returns True if the step
        was skipped (None with device_state)."""
        if grads is not None:
            self.table.set_grads(grads)
            self.norm_table.set_grads(grads)
        clip, hps = self.hyper[0]["max_grad_norm"], self._hypers()
        if self.state is not None:
            adam = [AdamHyper(max_grad_norm=clip)]
            if allreduce is None:
                zero_multi_norm_decide_dev(self.norm_table, adam, self.state, self.sqnorm, self.overflow, self.d_coefs,
                                           self.norm_workspace, self.tensor_sqnorm, unscaled)
            else:
                zero_multi_unscale_norm_overflow_dev(self.norm_table, self.state, self.sqnorm, self.overflow,
                                                     self.norm_workspace, self.tensor_sqnorm, unscaled)
                allreduce(self.sqnorm, self.overflow)
                zero_multi_decide_dev(adam, self.state, self.overflow, self.d_coefs, unscaled)
            zero_multi_momentum_step_coef(self.table, hps, self.d_coefs, self.sqnorm, self.overflow)
            self._apply(hps)
            return None
        inv = 1.0 if unscaled else 1.0 / self.scaler.scale
        zero_multi_unscale_norm_overflow(self.norm_table, inv, self.sqnorm, self.overflow, self.norm_workspace,
                                         self.tensor_sqnorm)
        if allreduce is not None:
            allreduce(self.sqnorm, self.overflow)
        zero_multi_momentum_step(self.table, hps, inv, clip, self.sqnorm, self.overflow)
        self._apply(hps)
        self._flag_host.copy_(self.overflow, non_blocking=True)
        self._flag_ready.record()
        self._flag_ready.synchronize()
        skip = zero_loss_scaler_update(self.scaler, bool(self._flag_host.item()))
        if not skip:
            self.t += 1
        return skip

    def _apply(self, hps) -> None:
        zero_multi_orthogonalize(self.table, self.workspace, self.coefs, self.eps, self.overflow)
        zero_multi_muon_update(self.table, hps, self.overflow)

    def release_grads(self) -> None:
        """MultiAdam.release_grads."""
        self.table.release_grads()
        self.norm_table.release_grads()

    def read_state(self):
        """device_state: copy the state to the host (waits for the steps enqueued
        so far), refresh self.t and self.scaler from it and return it."""
        st = self.state.read()
        self.t = st.applied
        self.scaler.s = type(self.scaler.s).from_buffer_copy(bytes(st.scaler))
        return st
