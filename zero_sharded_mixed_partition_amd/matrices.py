"""A step by orthogonalised momentum over a list of matrices: the table that
describes the list, the momentum pass, the orthogonalisation of its updates by a
Newton-Schulz iteration, and the update of the masters by the result.

    MatrixTable(updates, orthos=None, momentums=None, grads=None, masters=None, params_out=None, scales=None, groups=None)
    zero_multi_momentum_step(table, hps, inv_loss_scale, max_grad_norm, global_sqnorm, global_overflow)
    zero_multi_momentum_step_coef(table, hps, d_coef, global_sqnorm, global_overflow)
    zero_multi_orthogonalize_workspace_bytes(table) -> int
    zero_multi_orthogonalize(table, workspace, coefs, eps, global_overflow)
    zero_multi_muon_update(table, hps, global_overflow)
"""
import ctypes
from typing import Optional, Sequence

import torch

from . import _lib as _L
from . import _stream, dtype_code, zero_adam_coef_bytes, zero_muon_params
from .moments8 import _buf, _current_device
from .multi import MAX_GROUPS, TensorTable, _where

# five quintic steps that take singular values of [0.002, 1] to [0.68, 1.21]
ORTHO_COEFS = ((3.4445, -4.7750, 2.0315),) * 5


class MuonHyper:
    """Hyperparameters of one step (all double at the ABI)."""

    def __init__(self, lr=2e-2, momentum=0.95, weight_decay=0.0, nesterov=True):
        self.lr, self.momentum, self.weight_decay, self.nesterov = lr, momentum, weight_decay, nesterov

    def c(self) -> zero_muon_params:
        return zero_muon_params(float(self.lr), float(self.momentum), float(self.weight_decay),
                                1 if self.nesterov else 0, 0)


class MatrixTable(TensorTable):
    """The table of a list of matrices (zero_matrix_table_build), which lives and
    follows streams and graphs as a TensorTable.  Entries have two dimensions
    (rows, columns), or three: a batch of matrices.  All lists give one tensor
    per entry; those that no call needs may be left out:

        momentums   float32       the momentum pass, with grads and updates
        grads       fp16, bf16 or fp32
        updates     fp16, bf16 or fp32: written by the momentum pass, read by the
                    orthogonalisation
        orthos      fp16 or bf16: written by the orthogonalisation, read by the
                    update.  None: updates' own memory, if all are of 16 bits
        masters     float32       the update
        params_out  fp16 or bf16 copies of the masters (None entries: no copy)

    scales: each matrix's factor of the learning rate (default 1); groups: its
    hyperparameter group (default 0)."""

    _builder = "zero_matrix_table_build"

    def __init__(self, updates=None, orthos=None, momentums=None, grads=None, masters=None, params_out=None,
                 scales: Optional[Sequence[float]] = None, groups: Optional[Sequence[int]] = None):
        if orthos is None and updates is not None:
            updates = orthos = list(updates)
            if any(x.dtype == torch.float32 for x in updates):
                orthos = None                      # an update of 32 bits is no place for a result of 16
        lists = dict(updates=updates, orthos=orthos, momentums=momentums, grads=grads, masters=masters,
                     params_out=params_out, scales=scales, groups=groups)
        lists = {k: list(x) for k, x in lists.items() if x is not None}
        shaped = next((lists[k] for k in ("updates", "orthos", "masters") if k in lists), None)
        if shaped is None:
            raise ValueError("updates, orthos or masters expected")
        for name, x in lists.items():
            if len(x) != len(shaped):
                raise ValueError(f"{name} has {len(x)} entries, {len(shaped)} expected")
        self.shapes = [tuple(x.shape) for x in shaped]
        for i, shape in enumerate(self.shapes):
            if len(shape) not in (2, 3):
                raise ValueError(f"entry {i}: a matrix or a batch of matrices expected, got shape {shape}")
            for name in ("updates", "orthos", "momentums", "grads", "masters", "params_out"):
                x = lists.get(name)
                if x is not None and x[i] is not None and tuple(x[i].shape) != shape:
                    raise ValueError(f"{name}[{i}]: shape {tuple(x[i].shape)}, {shape} expected")
        self.state_bits, self.n_tensors = 0, len(shaped)
        get = lists.get
        self.updates, self.orthos, self.momentums = get("updates"), get("orthos"), get("momentums")
        self.masters, self.params_out = get("masters"), get("params_out")
        self.scales, self.groups = get("scales"), get("groups")
        self.n_groups = 1 + max(self.groups) if self.groups else 1
        self._ready, self._kept = None, []
        self._has_grads = "grads" in lists
        grads = lists.get("grads", [])
        self._describe(shaped)
        self._build(grads, _where(grads))

    def set_grads(self, grads) -> None:
        """TensorTable.set_grads; gradients of the matrices' shapes."""
        if not self._has_grads:
            raise ValueError("the table was built without gradients")
        for i, (g, shape) in enumerate(zip(grads, self.shapes)):
            if tuple(g.shape) != shape:
                raise ValueError(f"grads[{i}]: shape {tuple(g.shape)}, {shape} expected")
        super().set_grads(grads)

    def release_grads(self) -> None:
        """TensorTable.release_grads; nothing where the table has no gradients."""
        if self._has_grads:
            super().release_grads()

    def _describe(self, shaped) -> None:
        self._c = (_L.zero_matrix * max(1, self.n_tensors))()
        self._index = shaped[0].get_device() if shaped and hasattr(shaped[0], "get_device") else -1
        self._numels = [x.numel() for x in shaped]
        for i, (n, shape) in enumerate(zip(self._numels, self.shapes)):
            t = self._c[i]
            t.batch, t.rows, t.cols = (1,) * (3 - len(shape)) + shape
            t.scale = 1.0 if self.scales is None else float(self.scales[i])
            t.group = 0 if self.groups is None else int(self.groups[i])
            for field, name, dtype in (("master", "masters", torch.float32), ("momentum", "momentums", torch.float32),
                                       ("update", "updates", None), ("ortho", "orthos", None),
                                       ("param_out", "params_out", None)):
                x = getattr(self, name)
                if x is None or x[i] is None:
                    continue
                setattr(t, field, _buf(x[i], dtype, 0, f"{name}[{i}]", self._index, n))
                if dtype is None:
                    setattr(t, field.replace("_out", "") + "_dtype", dtype_code(x[i]))

    def _describe_grads(self, grads) -> None:
        for i, (g, n) in enumerate(zip(grads, self._numels)):
            t = self._c[i]
            t.grad, t.grad_dtype = _buf(g, None, 0, f"grads[{i}]", self._index, n), dtype_code(g)

    def _write(self, where, capacity: int, size, dev_size) -> int:
        return _L.lib().zero_matrix_table_build(self._c, self.n_tensors, where, capacity, ctypes.byref(size),
                                                ctypes.byref(dev_size))


def _params(hps):
    if not 1 <= len(hps) <= MAX_GROUPS:
        raise ValueError(f"1 to {MAX_GROUPS} hyperparameter sets expected, got {len(hps)}")
    return (zero_muon_params * len(hps))(*[h.c() for h in hps])


def _scalars(dev, global_sqnorm, global_overflow):
    return (_buf(global_sqnorm, torch.float64, 8, "global_sqnorm", dev),
            _buf(global_overflow, torch.int32, 4, "global_overflow", dev))


def zero_multi_momentum_step(table: MatrixTable, hps: Sequence[MuonHyper], inv_loss_scale: float = 1.0,
                             max_grad_norm: float = 0.0, global_sqnorm=None, global_overflow=None, stream=None) -> None:
    """Enqueue the momentum pass: momentums <- the exponential average of the
    unscaled and clipped gradients, updates <- it or its Nesterov form."""
    arr, dev = _params(hps), _current_device()
    _L.check(_L.lib().zero_multi_momentum_step(*table._ptrs(dev, stream), arr, len(hps), float(inv_loss_scale),
                                               float(max_grad_norm), *_scalars(dev, global_sqnorm, global_overflow),
                                               _stream(stream, dev)), "zero_multi_momentum_step")


def zero_multi_momentum_step_coef(table: MatrixTable, hps: Sequence[MuonHyper], d_coef, global_sqnorm,
                                  global_overflow=None, stream=None) -> None:
    """zero_multi_momentum_step with the loss scale and the clip norm from a
    coefficient block in device memory (zero_multi_decide_dev)."""
    arr, dev = _params(hps), _current_device()
    _L.check(_L.lib().zero_multi_momentum_step_coef(*table._ptrs(dev, stream), arr, len(hps),
                                                    _buf(d_coef, None, zero_adam_coef_bytes(), "d_coef", dev),
                                                    *_scalars(dev, global_sqnorm, global_overflow),
                                                    _stream(stream, dev)), "zero_multi_momentum_step_coef")


def zero_multi_orthogonalize_workspace_bytes(table: MatrixTable) -> int:
    return int(_L.lib().zero_multi_orthogonalize_workspace_bytes(table.host.data_ptr()))


def zero_multi_orthogonalize(table: MatrixTable, workspace, coefs=ORTHO_COEFS, eps: float = 1e-7, global_overflow=None,
                             stream=None) -> None:
    """Enqueue the orthogonalisation of every matrix of the list: orthos <- X
    after the steps X <- a X + (b X X^T + c (X X^T)^2) X for the (a, b, c) of
    coefs, from X = update / max(its Frobenius norm, eps)."""
    steps = [tuple(float(x) for x in step) for step in coefs]
    if any(len(step) != 3 for step in steps):
        raise ValueError("coefs: three numbers per step expected")
    flat = [x for step in steps for x in step]
    dev = _current_device()
    _L.check(_L.lib().zero_multi_orthogonalize(*table._ptrs(dev, stream), (ctypes.c_double * max(1, len(flat)))(*flat),
                                               len(steps), float(eps),
                                               _buf(global_overflow, torch.int32, 4, "global_overflow", dev),
                                               _buf(workspace, None, 0, "workspace", dev),
                                               workspace.numel() * workspace.element_size(), _stream(stream, dev)),
             "zero_multi_orthogonalize")


def zero_multi_muon_update(table: MatrixTable, hps: Sequence[MuonHyper], global_overflow=None, stream=None) -> None:
    """Enqueue the update: masters <- masters (1 - lr weight_decay) - lr scale ortho,
    and the copies."""
    arr, dev = _params(hps), _current_device()
    _L.check(_L.lib().zero_multi_muon_update(*table._ptrs(dev, stream), arr, len(hps),
                                             _buf(global_overflow, torch.int32, 4, "global_overflow", dev),
                                             _stream(stream, dev)), "zero_multi_muon_update")
