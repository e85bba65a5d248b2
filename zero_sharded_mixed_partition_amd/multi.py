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

import torch

from . import _lib as _L
from . import (AdamHyper, StepState, _hyper, _stream, dtype_code, zero_adam_coef_bytes, zero_adam_hyper,
               zero_adam_params)
from .moments8 import _buf, _codes_bytes, _current_device, _scales_bytes, _seed

MAX_GROUPS = 16


def _f32_bytes(n: int) -> int:
    return 4 * n


def _where(grads):
    return [(g.data_ptr(), g.dtype, g.numel(), g.is_contiguous()) for g in grads]


class TensorTable:
    """The list's table (zero_multi_table_build): a host part and its device
    copy.  Holds references to the tensors (the gradients: until release_grads)
    and describes their addresses: that one is resized or given other storage
    afterwards is not seen.  A recorded graph reads the device copy: keep the table
    as long as the graph.  groups:
    hyperparameter group per tensor (default 0).  state_bits 8: exp_avgs and
    exp_avg_sqs are the tensors' moments8 and scales8 (uint8)."""

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
        own = lambda x: None if x is None else list(x)  # noqa: E731
        self.masters, self.exp_avgs, self.exp_avg_sqs = own(masters), own(exp_avgs), own(exp_avg_sqs)
        self.params_out, self.groups = own(params_out), own(groups)
        self.n_groups = 1 + max(self.groups) if self.groups else 1
        self._ready = None                     # the copy to the device has run
        self._kept = []                        # tables that recorded graphs read, and their gradients
        self._describe(grads)
        self._build(grads, _where(grads))

    @classmethod
    def of_grads(cls, grads) -> "TensorTable":
        """A table for the norm pass alone."""
        return cls(None, None, None, grads, state_bits=0)

    def set_grads(self, grads) -> None:
        """Describe the list anew with other gradient tensors of the same lengths
        (a no-op if they lie where the present ones do).  The new device copy is
        enqueued on the current stream, and torch streams that use the table wait
        for it; the old one lives until every torch stream that read it has passed
        (a raw stream handle is the caller's to wait for, and so is the copy if a
        graph is recorded on another stream: torch.cuda.graph synchronizes first).
        A graph that torch recorded with the table keeps reading the old gradients
        (which the table then keeps alive, with their description): record it again."""
        if len(grads) != self.n_tensors:
            raise ValueError(f"{len(grads)} gradients for {self.n_tensors} tensors")
        key = _where(grads)
        if key != self._grad_key:
            old, captured = (self.host, self.device, self.grads), self._captured
            self._build(grads, key)
            if captured:
                self._kept.append(old)
        elif self.grads is None:
            self.grads = list(grads)

    def release_grads(self) -> None:
        """Let go of the gradient tensors, once the calls that read them are
        enqueued: else they stay allocated until set_grads names others.  The table
        then needs set_grads before its next use (a no-op again if the allocator
        put the new ones in the same place).  Gradients that a recorded graph reads
        are kept.  As for any torch tensor, calls on another stream than the
        gradients' own need record_stream on them first."""
        if self._captured and self.grads is not None:
            self._kept.append(self.grads)
        self.grads = None

    def _describe(self, grads) -> None:
        """The C descriptions of the whole list."""
        self._c = (_L.zero_tensor * max(1, self.n_tensors))()
        bits = self.state_bits
        self._index = grads[0].get_device() if grads and hasattr(grads[0], "get_device") else -1
        self._numels = [g.numel() for g in grads]
        if not bits:
            return
        kinds = (torch.uint8, _codes_bytes, _scales_bytes) if bits == 8 else (torch.float32, _f32_bytes, _f32_bytes)
        for i, n in enumerate(self._numels):
            t = self._c[i]
            t.master = _buf(self.masters[i], torch.float32, 4 * n, f"masters[{i}]", self._index, n)
            t.exp_avg = _buf(self.exp_avgs[i], kinds[0], kinds[1](n), f"exp_avgs[{i}]", self._index)
            t.exp_avg_sq = _buf(self.exp_avg_sqs[i], kinds[0], kinds[2](n), f"exp_avg_sqs[{i}]", self._index)
            p = None if self.params_out is None else self.params_out[i]
            if p is not None:
                t.param_out, t.param_dtype = _buf(p, None, 2 * n, f"params_out[{i}]", self._index, n), dtype_code(p)
            if self.groups is not None:
                t.group = int(self.groups[i])

    def _build(self, grads, key) -> None:
        """The table for these gradients, the rest of the list being described."""
        arr, bits, index = self._c, self.state_bits, self._index
        for i, (g, n) in enumerate(zip(grads, self._numels)):
            t = arr[i]
            t.grad, t.numel, t.grad_dtype = _buf(g, None, 0, f"grads[{i}]", index, n), n, dtype_code(g)
        size, dev_size = ctypes.c_size_t(), ctypes.c_size_t()
        build = _L.lib().zero_multi_table_build
        st = build(arr, self.n_tensors, bits, None, 0, ctypes.byref(size), ctypes.byref(dev_size))
        if st != _L.ZERO_ENOSPC:
            _L.check(st, "zero_multi_table_build")
        on_gpu = index >= 0
        if on_gpu and torch.cuda.is_current_stream_capturing():
            raise RuntimeError("a table cannot be built while its stream records a graph")
        # pinned: the copy to the device needs no wait, and torch's host allocator
        # hands the memory out again only after the copy has run
        host = torch.empty(size.value, dtype=torch.uint8, pin_memory=on_gpu)
        _L.check(build(arr, self.n_tensors, bits, host.data_ptr(), size.value, ctypes.byref(size),
                       ctypes.byref(dev_size)), "zero_multi_table_build")
        self.grads, self.host = list(grads), host
        self._grad_key = key
        self.device = host[:dev_size.value].to(torch.device("cuda", index), non_blocking=True) if on_gpu else None
        self._captured = False
        # raw handles of the streams that have read the device copy; its own needs no wait and no record
        self._streams = {_stream(None, index)} if on_gpu else set()
        if on_gpu:
            if self._ready is None:
                self._ready = torch.cuda.Event()
            self._ready.record(torch.cuda.current_stream(index))
        self._addresses = self.host.data_ptr(), None if self.device is None else self.device.data_ptr()

    def _ptrs(self, current: int, stream):
        if self.grads is None:
            raise ValueError("the table's gradients were released: set_grads first")
        if self._index < 0:
            return self._addresses
        if self._index != current:
            raise ValueError(f"the table's tensors are on cuda:{self._index}, the current device is cuda:{current}")
        if not self._captured:
            self._captured = torch.cuda.is_current_stream_capturing()
        if not isinstance(stream, int):
            raw = _stream(stream, current)
            if raw not in self._streams:
                # the stream waits for the device copy, and the allocator keeps it
                # until the stream has passed the calls that read it
                used = torch.cuda.current_stream() if stream is None else stream
                self.device.record_stream(used)
                recording = self._ready is not None and torch.cuda.is_current_stream_capturing()
                if not recording:                     # a recording stream can wait for nothing outside its graph
                    self._streams.add(raw)
                    if self._ready is not None:
                        used.wait_event(self._ready)
        return self._addresses


def zero_multi_norm_workspace_bytes(table: TensorTable) -> int:
    return int(_L.lib().zero_multi_norm_workspace_bytes(table.host.data_ptr()))


def _norm_args(table, sqnorm, overflow, tensor_sqnorm, workspace, stream):
    dev = _current_device()
    return (dev, table._ptrs(dev, stream),
            (_buf(sqnorm, torch.float64, 8, "sqnorm", dev), _buf(overflow, torch.int32, 4, "overflow", dev),
             _buf(tensor_sqnorm, torch.float64, 8 * table.n_tensors, "tensor_sqnorm", dev)),
            (_buf(workspace, None, 0, "workspace", dev), workspace.numel() * workspace.element_size()))


def zero_multi_unscale_norm_overflow(table: TensorTable, inv_loss_scale: float, sqnorm, overflow, workspace,
                                     tensor_sqnorm=None, stream=None) -> None:
    """Enqueue the norm pass over the list's gradients: sqnorm (float64 [1]),
    overflow (int32 [1]) and, if given, each tensor's own sum of squares
    (tensor_sqnorm, float64 [n_tensors])."""
    dev, tab, out, ws = _norm_args(table, sqnorm, overflow, tensor_sqnorm, workspace, stream)
    _L.check(_L.lib().zero_multi_unscale_norm_overflow(*tab, float(inv_loss_scale), *out, *ws, _stream(stream, dev)),
             "zero_multi_unscale_norm_overflow")


def zero_multi_unscale_norm_overflow_dev(table: TensorTable, state: StepState, sqnorm, overflow, workspace,
                                         tensor_sqnorm=None, unscaled: bool = False, stream=None) -> None:
    """The norm pass with the loss scale from the device state; unscaled: the
    gradients are already unscaled."""
    dev, tab, out, ws = _norm_args(table, sqnorm, overflow, tensor_sqnorm, workspace, stream)
    _L.check(_L.lib().zero_multi_unscale_norm_overflow_dev(*tab, 1 if unscaled else 0, state.ptr(), *out, *ws,
                                                           _stream(stream, dev)),
             "zero_multi_unscale_norm_overflow_dev")


def _hypers(hps):
    if not 1 <= len(hps) <= MAX_GROUPS:
        raise ValueError(f"1 to {MAX_GROUPS} hyperparameter sets expected, got {len(hps)}")
    return (zero_adam_hyper * len(hps))(*[_hyper(h) for h in hps])


def _coefs_ptr(d_coefs, n_groups: int, dev: int) -> Optional[int]:
    return _buf(d_coefs, None, n_groups * zero_adam_coef_bytes(), "d_coefs", dev)


def zero_multi_norm_decide_dev(table: TensorTable, hps: Sequence[AdamHyper], state: StepState, sqnorm, overflow,
                               d_coefs, workspace, tensor_sqnorm=None, unscaled: bool = False, stream=None) -> None:
    """The norm pass of a single rank, whose last kernel also makes the step's
    decision: one coefficient block per set into d_coefs, the state advanced.  A
    recorded call keeps the hyperparameters it was recorded with."""
    dev, tab, out, ws = _norm_args(table, sqnorm, overflow, tensor_sqnorm, workspace, stream)
    _L.check(_L.lib().zero_multi_norm_decide_dev(*tab, 1 if unscaled else 0, _hypers(hps), len(hps), state.ptr(), *out,
                                                 _coefs_ptr(d_coefs, len(hps), dev), *ws, _stream(stream, dev)),
             "zero_multi_norm_decide_dev")


def zero_multi_decide_dev(hps: Sequence[AdamHyper], state: StepState, global_overflow, d_coefs,
                          unscaled: bool = False, stream=None) -> None:
    """The decision alone: d_coefs <- the blocks of step applied + 1, the state
    advanced by the flag."""
    dev = _current_device()
    _L.check(_L.lib().zero_multi_decide_dev(_hypers(hps), len(hps), 1 if unscaled else 0, state.ptr(),
                                            _buf(global_overflow, torch.int32, 4, "global_overflow", dev),
                                            _coefs_ptr(d_coefs, len(hps), dev), _stream(stream, dev)), "zero_multi_decide_dev")


def zero_multi_adam_step(table: TensorTable, hps: Sequence[AdamHyper], global_sqnorm=None, global_overflow=None,
                         seed: int = 0, stream=None) -> None:
    """Enqueue the update of every tensor of the list with hps[group]; seed keys
    the rounding of 8-bit moments."""
    if not 1 <= len(hps) <= MAX_GROUPS:
        raise ValueError(f"1 to {MAX_GROUPS} hyperparameter sets expected, got {len(hps)}")
    dev = _current_device()
    arr = (zero_adam_params * len(hps))(*[h.c() for h in hps])
    _L.check(_L.lib().zero_multi_adam_step(*table._ptrs(dev, stream), arr, len(hps), _seed(seed),
                                           _buf(global_sqnorm, torch.float64, 8, "global_sqnorm", dev),
                                           _buf(global_overflow, torch.int32, 4, "global_overflow", dev), _stream(stream, dev)),
             "zero_multi_adam_step")


def zero_multi_adam_step_coef(table: TensorTable, d_coefs, n_groups: int, global_sqnorm, global_overflow=None,
                              d_step=None, seed: int = 0, stream=None) -> None:
    """zero_multi_adam_step with the coefficient blocks read from device memory
    d_coefs and, for 8-bit moments, the step that keys the rounding from d_step
    (int64 [1])."""
    dev = _current_device()
    _L.check(_L.lib().zero_multi_adam_step_coef(*table._ptrs(dev, stream), _coefs_ptr(d_coefs, n_groups, dev), n_groups, _seed(seed),
                                                _buf(d_step, torch.int64, 8, "d_step", dev),
                                                _buf(global_sqnorm, torch.float64, 8, "global_sqnorm", dev),
                                                _buf(global_overflow, torch.int32, 4, "global_overflow", dev),
                                                _stream(stream, dev)), "zero_multi_adam_step_coef")
