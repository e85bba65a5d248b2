"""The shard's step with its moments in 8 bits, and their conversion.

    zero_moments8_bytes(n), zero_scales8_bytes(n) -> int
    zero_moments8_pack(moments8, scales8, exp_avg, exp_avg_sq)
    zero_moments8_unpack(exp_avg, exp_avg_sq, moments8, scales8)
    zero_shard_adam8_step(master, moments8, scales8, grad, param_out, hp, global_sqnorm, global_overflow, seed)
    zero_shard_adam8_step_coef(master, moments8, scales8, grad, param_out, d_coef, d_step, ...)

The format (blocks of 32, e4m3 codes of exp_avg and of the square root of
exp_avg_sq, one power of two per block and moment, stochastic rounding keyed
by the seed and the step) is described in include/zero_shard.h.
"""
import ctypes
from typing import Optional

from . import _lib as _L
from . import (AdamHyper, _coef_ptr, _dev, _grad_ptr, _stream, _typed, dtype_code)


def zero_moments8_bytes(n: int) -> int:
    return int(_L.lib().zero_moments8_bytes(int(n)))


def zero_scales8_bytes(n: int) -> int:
    return int(_L.lib().zero_scales8_bytes(int(n)))


def _same_device(*tensors) -> None:
    """The kernels run on the current device's stream: tensors that say where
    they live must live there."""
    import torch
    found = {t.device for t in tensors if hasattr(t, "device") and not isinstance(t, int)}
    if len(found) > 1:
        raise ValueError(f"tensors on different devices: {sorted(map(str, found))}")
    for d in found:
        if d.type == "cuda" and d.index != torch.cuda.current_device():
            raise ValueError(f"tensors on {d}, the current device is cuda:{torch.cuda.current_device()}")


def _seed(seed: int) -> int:
    return int(seed) & 0xFFFFFFFFFFFFFFFF


def _bytes8(t, nbytes: int, what: str) -> Optional[int]:
    if t is not None and not isinstance(t, int) and str(t.dtype) != "torch.uint8":
        raise ValueError(f"{what}: torch.uint8 tensor expected, got {t.dtype}")
    return _dev(t, nbytes, what)


def _f32(t, n: int, what: str) -> Optional[int]:
    if t is not None and not isinstance(t, int) and str(t.dtype) != "torch.float32":
        raise ValueError(f"{what}: torch.float32 tensor expected, got {t.dtype}")
    return _dev(t, 4 * n, what)


def _step8_ptrs(master, moments8, scales8, grad, gd: int, param_out, n: int):
    if not isinstance(master, int):
        for t in (grad,) + (() if param_out is None else (param_out,)):
            if not isinstance(t, int) and t.numel() != n:
                raise ValueError("shard tensors differ in length")
    _same_device(master, moments8, scales8, grad, param_out)
    return (_f32(master, n, "master"), _bytes8(moments8, zero_moments8_bytes(n), "moments8"),
            _bytes8(scales8, zero_scales8_bytes(n), "scales8"), _grad_ptr(grad, gd, n), _dev(param_out, 2 * n, "param_out"))


def zero_shard_adam8_step(master, moments8, scales8, grad, param_out, hp: AdamHyper, global_sqnorm=None,
                          global_overflow=None, seed: int = 0, grad_dtype: Optional[int] = None,
                          param_dtype: Optional[int] = None, n: Optional[int] = None, stream=None) -> None:
    """Enqueue the fused AdamW update with 8-bit moments on the current stream:
    moments8 and scales8 are uint8 tensors of at least zero_moments8_bytes(n)
    and zero_scales8_bytes(n) bytes; seed and hp.step key the rounding."""
    gd = dtype_code(grad if grad_dtype is None else grad_dtype)
    pd = 0 if param_out is None else dtype_code(param_out if param_dtype is None else param_dtype)
    n = master.numel() if n is None else n
    params = hp.c()
    pm, pc, ps, pg, pp = _step8_ptrs(master, moments8, scales8, grad, gd, param_out, n)
    _L.check(_L.lib().zero_shard_adam8_step(pm, pc, ps, pg, gd, pp, pd, n, ctypes.byref(params), _seed(seed),
                                            _typed(global_sqnorm, "float64", 1, "global_sqnorm"),
                                            _typed(global_overflow, "int32", 1, "global_overflow"), _stream(stream)),
             "zero_shard_adam8_step")


def zero_shard_adam8_step_coef(master, moments8, scales8, grad, param_out, d_coef, d_step, global_sqnorm,
                               global_overflow=None, seed: int = 0, grad_dtype: Optional[int] = None,
                               param_dtype: Optional[int] = None, n: Optional[int] = None, stream=None) -> None:
    """zero_shard_adam8_step with the coefficient block read from device memory
    d_coef and the step that keys the rounding from d_step (int64 [1])."""
    gd = dtype_code(grad if grad_dtype is None else grad_dtype)
    pd = 0 if param_out is None else dtype_code(param_out if param_dtype is None else param_dtype)
    n = master.numel() if n is None else n
    pm, pc, ps, pg, pp = _step8_ptrs(master, moments8, scales8, grad, gd, param_out, n)
    _L.check(_L.lib().zero_shard_adam8_step_coef(pm, pc, ps, pg, gd, pp, pd, n, _coef_ptr(d_coef), _seed(seed),
                                                 _typed(d_step, "int64", 1, "d_step"),
                                                 _typed(global_sqnorm, "float64", 1, "global_sqnorm"),
                                                 _typed(global_overflow, "int32", 1, "global_overflow"),
                                                 _stream(stream)), "zero_shard_adam8_step_coef")


def zero_moments8_pack(moments8, scales8, exp_avg, exp_avg_sq, n: Optional[int] = None, stream=None) -> None:
    """Codes and block scales of fp32 moments, rounded to nearest."""
    n = exp_avg.numel() if n is None else n
    _same_device(moments8, scales8, exp_avg, exp_avg_sq)
    _L.check(_L.lib().zero_moments8_pack(_bytes8(moments8, zero_moments8_bytes(n), "moments8"),
                                         _bytes8(scales8, zero_scales8_bytes(n), "scales8"),
                                         _f32(exp_avg, n, "exp_avg"), _f32(exp_avg_sq, n, "exp_avg_sq"), n,
                                         _stream(stream)), "zero_moments8_pack")


def zero_moments8_unpack(exp_avg, exp_avg_sq, moments8, scales8, n: Optional[int] = None, stream=None) -> None:
    """fp32 moments from their codes and block scales."""
    n = exp_avg.numel() if n is None else n
    _same_device(moments8, scales8, exp_avg, exp_avg_sq)
    _L.check(_L.lib().zero_moments8_unpack(_f32(exp_avg, n, "exp_avg"), _f32(exp_avg_sq, n, "exp_avg_sq"),
                                           _bytes8(moments8, zero_moments8_bytes(n), "moments8"),
                                           _bytes8(scales8, zero_scales8_bytes(n), "scales8"), n, _stream(stream)),
             "zero_moments8_unpack")
