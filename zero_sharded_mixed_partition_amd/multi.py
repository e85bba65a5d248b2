"""The step over a list of tensors: the table that describes the list, the norm
pass over its gradients and the update of all of it in one launch.

    TensorTable(masters, exp_avgs, exp_avg_sqs, grads, params_out=None, groups=None, state_bits=32)
    TensorTable.of_grads(grads)
    zero_multi_norm_workspace_bytes(table) -> int
    zero_multi_unscale_norm_overflow(table, inv_loss_scale, sqnorm, overflow, workspace, tensor_sqnorm=None)
    zero_multi_adam_step(table, hps, global_sqnorm, global_overflow, seed=0)
    zero_multi_adam_step_coef(table, d_coefs, n_groups, global_sqnorm, global_overflow, d_step=None, seed=0)

and their *_dev forms with the loss scaler and step counter in device memory.
"""
import ctypes
from typing import Optional, Sequence

from . import _lib as _L
from . import (AdamHyper, StepState, _dev, _hyper, _ptr, _stream, _typed, dtype_code, zero_adam_coef_bytes,
               zero_adam_hyper, zero_adam_params)
from .moments8 import _bytes8, _f32, _same_device, _seed, zero_moments8_bytes, zero_scales8_bytes

MAX_GROUPS = 16


def _upload(host, device):
    """A device copy of host bytes, enqueued on the current stream.  The pinned
    source returns to torch's host allocator, which hands it out again only
    after the copy has run."""
    import torch
    pinned = torch.empty(host.numel(), dtype=torch.uint8, pin_memory=True)
    pinned.copy_(host)
    return pinned.to(device, non_blocking=True)


class TensorTable:
    """The list's table (zero_multi_table_build): a host part and its device
    copy.  Holds references to the tensors.  groups: hyperparameter group per
    tensor (default 0).  state_bits 8: exp_avgs and exp_avg_sqs are the
    tensors' moments8 and scales8 (uint8)."""

    def __init__(self, masters, exp_avgs, exp_avg_sqs, grads, params_out=None, groups: Optional[Sequence[int]] = None,
                 state_bits: int = 32):
        n = len(grads)
        lists = dict(masters=masters, exp_avgs=exp_avgs, exp_avg_sqs=exp_avg_sqs)
        if state_bits == 0:
            lists = {}
        if params_out is not None:
            lists["params_out"] = params_out
        if groups is not None:
            lists["groups"] = groups
        for name, x in lists.items():
            if len(x) != n:
                raise ValueError(f"{name} has {len(x)} entries, grads {n}")
        if state_bits not in (0, 8, 32):
            raise ValueError(f"state_bits must be 32 or 8, got {state_bits}")
        self.state_bits, self.n_tensors = state_bits, n
        self.masters, self.exp_avgs, self.exp_avg_sqs = masters, exp_avgs, exp_avg_sqs
        self.params_out, self.groups = params_out, None if groups is None else list(groups)
        self.n_groups = 1 + max(self.groups) if self.groups else 1
        self._build(grads)

    @classmethod
    def of_grads(cls, grads) -> "TensorTable":
        """A table for the norm pass alone."""
        return cls(None, None, None, grads, state_bits=0)

    def set_grads(self, grads) -> None:
        """Describe the list anew with other gradient tensors (a no-op if they
        lie where the present ones do).  The new device copy is enqueued on the
        current stream; a recorded graph keeps the old one, so recording again
        is the caller's part."""
        if len(grads) != self.n_tensors:
            raise ValueError(f"{len(grads)} gradients for {self.n_tensors} tensors")
        now = tuple((g.data_ptr(), g.dtype, g.numel()) for g in grads)
        if now != self._grad_key:
            self._build(grads)

    def _build(self, grads) -> None:
        import torch
        self.grads = list(grads)
        self._grad_key = tuple((g.data_ptr(), g.dtype, g.numel()) for g in self.grads)
        arr = (_L.zero_tensor * max(1, self.n_tensors))()
        device = None
        for i, g in enumerate(self.grads):
            n = g.numel()
            t = arr[i]
            t.grad, t.numel, t.grad_dtype = _ptr(g), n, dtype_code(g)
            tensors = [g]
            if self.state_bits:
                m, a, b = self.masters[i], self.exp_avgs[i], self.exp_avg_sqs[i]
                if m.numel() != n:
                    raise ValueError(f"tensor {i}: master has {m.numel()} elements, grad {n}")
                t.master = _f32(m, n, f"masters[{i}]")
                if self.state_bits == 8:
                    t.exp_avg = _bytes8(a, zero_moments8_bytes(n), f"exp_avgs[{i}]")
                    t.exp_avg_sq = _bytes8(b, zero_scales8_bytes(n), f"exp_avg_sqs[{i}]")
                else:
                    t.exp_avg, t.exp_avg_sq = _f32(a, n, f"exp_avgs[{i}]"), _f32(b, n, f"exp_avg_sqs[{i}]")
                tensors += [m, a, b]
                p = None if self.params_out is None else self.params_out[i]
                if p is not None:
                    t.param_out, t.param_dtype = _dev(p, 2 * n, f"params_out[{i}]"), dtype_code(p)
                    tensors.append(p)
                t.group = 0 if self.groups is None else int(self.groups[i])
            for x in tensors:
                if hasattr(x, "device"):
                    if device is not None and x.device != device:
                        raise ValueError(f"tensor {i}: on {x.device}, others on {device}")
                    device = x.device
        size, dev_size = ctypes.c_size_t(), ctypes.c_size_t()
        st = _L.lib().zero_multi_table_build(arr, self.n_tensors, self.state_bits, None, 0, ctypes.byref(size),
                                             ctypes.byref(dev_size))
        if st != _L.ZERO_ENOSPC:
            _L.check(st, "zero_multi_table_build")
        self.host = torch.empty(size.value, dtype=torch.uint8)
        _L.check(_L.lib().zero_multi_table_build(arr, self.n_tensors, self.state_bits, self.host.data_ptr(), size.value,
                                                 ctypes.byref(size), ctypes.byref(dev_size)), "zero_multi_table_build")
        self.device = None
        if device is not None and device.type == "cuda":
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError("a table cannot be built while its stream records a graph")
            self.device = _upload(self.host[:dev_size.value], device)

    def _ptrs(self):
        if self.device is not None:
            _same_device(self.device)
        return self.host.data_ptr(), None if self.device is None else self.device.data_ptr()


def zero_multi_norm_workspace_bytes(table: TensorTable) -> int:
    return int(_L.lib().zero_multi_norm_workspace_bytes(table.host.data_ptr()))


def _norm_ptrs(table, sqnorm, overflow, tensor_sqnorm, workspace):
    return (_typed(sqnorm, "float64", 1, "sqnorm"), _typed(overflow, "int32", 1, "overflow"),
            _typed(tensor_sqnorm, "float64", table.n_tensors, "tensor_sqnorm"), _ptr(workspace),
            workspace.numel() * workspace.element_size())


def zero_multi_unscale_norm_overflow(table: TensorTable, inv_loss_scale: float, sqnorm, overflow, workspace,
                                     tensor_sqnorm=None, stream=None) -> None:
    """Enqueue the norm pass over the list's gradients: sqnorm (float64 [1]),
    overflow (int32 [1]) and, if given, each tensor's own sum of squares
    (tensor_sqnorm, float64 [n_tensors])."""
    host, dev = table._ptrs()
    sq, ov, per, ws, nb = _norm_ptrs(table, sqnorm, overflow, tensor_sqnorm, workspace)
    _L.check(_L.lib().zero_multi_unscale_norm_overflow(host, dev, float(inv_loss_scale), sq, ov, per, ws, nb,
                                                       _stream(stream)), "zero_multi_unscale_norm_overflow")


def zero_multi_unscale_norm_overflow_dev(table: TensorTable, state: StepState, sqnorm, overflow, workspace,
                                         tensor_sqnorm=None, unscaled: bool = False, stream=None) -> None:
    """The norm pass with the loss scale from the device state; unscaled: the
    gradients are already unscaled."""
    host, dev = table._ptrs()
    sq, ov, per, ws, nb = _norm_ptrs(table, sqnorm, overflow, tensor_sqnorm, workspace)
    _L.check(_L.lib().zero_multi_unscale_norm_overflow_dev(host, dev, 1 if unscaled else 0, state.ptr(), sq, ov, per,
                                                           ws, nb, _stream(stream)),
             "zero_multi_unscale_norm_overflow_dev")


def _hypers(hps):
    if not 1 <= len(hps) <= MAX_GROUPS:
        raise ValueError(f"1 to {MAX_GROUPS} hyperparameter sets expected, got {len(hps)}")
    return (zero_adam_hyper * len(hps))(*[_hyper(h) for h in hps])


def _coefs_ptr(d_coefs, n_groups: int) -> Optional[int]:
    return _dev(d_coefs, n_groups * zero_adam_coef_bytes(), "d_coefs")


def zero_multi_norm_decide_dev(table: TensorTable, hps: Sequence[AdamHyper], state: StepState, sqnorm, overflow,
                               d_coefs, workspace, tensor_sqnorm=None, unscaled: bool = False, stream=None) -> None:
    """The norm pass of a single rank, whose last kernel also makes the step's
    decision: one coefficient block per set into d_coefs, the state advanced."""
    host, dev = table._ptrs()
    sq, ov, per, ws, nb = _norm_ptrs(table, sqnorm, overflow, tensor_sqnorm, workspace)
    _L.check(_L.lib().zero_multi_norm_decide_dev(host, dev, 1 if unscaled else 0, _hypers(hps), len(hps), state.ptr(),
                                                 sq, ov, per, _coefs_ptr(d_coefs, len(hps)), ws, nb, _stream(stream)),
             "zero_multi_norm_decide_dev")


def zero_multi_decide_dev(hps: Sequence[AdamHyper], state: StepState, global_overflow, d_coefs,
                          unscaled: bool = False, stream=None) -> None:
    """The decision alone: d_coefs <- the blocks of step applied + 1, the state
    advanced by the flag."""
    _L.check(_L.lib().zero_multi_decide_dev(_hypers(hps), len(hps), 1 if unscaled else 0, state.ptr(),
                                            _typed(global_overflow, "int32", 1, "global_overflow"),
                                            _coefs_ptr(d_coefs, len(hps)), _stream(stream)), "zero_multi_decide_dev")


def zero_multi_adam_step(table: TensorTable, hps: Sequence[AdamHyper], global_sqnorm=None, global_overflow=None,
                         seed: int = 0, stream=None) -> None:
    """Enqueue the update of every tensor of the list with hps[group]; seed keys
    the rounding of 8-bit moments."""
    if not 1 <= len(hps) <= MAX_GROUPS:
        raise ValueError(f"1 to {MAX_GROUPS} hyperparameter sets expected, got {len(hps)}")
    host, dev = table._ptrs()
    arr = (zero_adam_params * len(hps))(*[h.c() for h in hps])
    _L.check(_L.lib().zero_multi_adam_step(host, dev, arr, len(hps), _seed(seed),
                                           _typed(global_sqnorm, "float64", 1, "global_sqnorm"),
                                           _typed(global_overflow, "int32", 1, "global_overflow"), _stream(stream)),
             "zero_multi_adam_step")


def zero_multi_adam_step_coef(table: TensorTable, d_coefs, n_groups: int, global_sqnorm, global_overflow=None,
                              d_step=None, seed: int = 0, stream=None) -> None:
    """zero_multi_adam_step with the coefficient blocks read from device memory
    d_coefs and, for 8-bit moments, the step that keys the rounding from d_step
    (int64 [1])."""
    host, dev = table._ptrs()
    _L.check(_L.lib().zero_multi_adam_step_coef(host, dev, _coefs_ptr(d_coefs, n_groups), n_groups, _seed(seed),
                                                _typed(d_step, "int64", 1, "d_step"),
                                                _typed(global_sqnorm, "float64", 1, "global_sqnorm"),
                                                _typed(global_overflow, "int32", 1, "global_overflow"),
                                                _stream(stream)), "zero_multi_adam_step_coef")
