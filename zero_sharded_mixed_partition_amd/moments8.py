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

import torch

from . import _lib as _L
from . import _ELEM_BYTES, AdamHyper, _stream, dtype_code, zero_adam_coef_bytes


def zero_moments8_bytes(n: int) -> int:
    return _L.lib().zero_moments8_bytes(int(n))


def zero_scales8_bytes(n: int) -> int:
    return _L.lib().zero_scales8_bytes(int(n))


def _current_device() -> int:
    return torch.cuda.current_device() if _on_gpu or _gpu_in_use() else -1


_on_gpu = False


def _gpu_in_use() -> bool:
    """Whether this process has a GPU context (remembered once it has)."""
    global _on_gpu
    _on_gpu = torch.cuda.is_initialized()
    return _on_gpu


def _buf(t, dtype, nbytes: int, what: str, device: int, exact: int = -1) -> Optional[int]:
    """Address of a device tensor after the checks: its dtype (None: any), at
    least nbytes bytes, contiguous, on the current device (whose stream the
    kernels run on), exact elements if given.  None and raw addresses are taken
    as they are."""
    if t is None or isinstance(t, int):
        return t
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{what}: {dtype} tensor expected, got {t.dtype}")
    n = t.numel()
    if exact >= 0 and n != exact:
        raise ValueError(f"{what}: {n} elements, {exact} expected")
    if not (t.get_device() == device if device >= 0 else t.is_cuda):
        raise ValueError(f"{what}: " + (f"on {t.device}, the current device is cuda:{device}" if device >= 0 and t.is_cuda
                                        else "device tensor expected"))
    if not t.is_contiguous():
        raise ValueError(f"{what}: contiguous tensor expected")
    if n * t.element_size() < nbytes:
        raise ValueError(f"{what}: {n * t.element_size()} bytes, the call accesses {nbytes}")
    return t.data_ptr()


def _codes_bytes(n: int) -> int:
    return 8 * -(-n // 4)


def _scales_bytes(n: int) -> int:
    return 2 * -(-n // 32)


def _seed(seed: int) -> int:
    return int(seed) & 0xFFFFFFFFFFFFFFFF


def _step8_ptrs(master, moments8, scales8, grad, gd: int, param_out, n: int, dev: int):
    exact = -1 if isinstance(master, int) else n
    return (_buf(master, torch.float32, 4 * n, "master", dev), _buf(moments8, torch.uint8, _codes_bytes(n), "moments8", dev),
            _buf(scales8, torch.uint8, _scales_bytes(n), "scales8", dev),
            _buf(grad, None, n * _ELEM_BYTES.get(gd, 0), "grad", dev, exact),
            _buf(param_out, None, 2 * n, "param_out", dev, exact))


def zero_shard_adam8_step(master, moments8, scales8, grad, param_out, hp: AdamHyper, global_sqnorm=None,
                          global_overflow=None, seed: int = 0, grad_dtype: Optional[int] = None,
                          param_dtype: Optional[int] = None, n: Optional[int] = None, stream=None) -> None:
    """Enqueue the fused AdamW update with 8-bit moments on the current stream:
    moments8 and scales8 are uint8 tensors of at least zero_moments8_bytes(n)
    and zero_scales8_bytes(n) bytes; seed and hp.step key the rounding."""
    gd = dtype_code(grad if grad_dtype is None else grad_dtype)
    pd = 0 if param_out is None else dtype_code(param_out if param_dtype is None else param_dtype)
    n = master.numel() if n is None else n
    params, dev = hp.c(), _current_device()
    pm, pc, ps, pg, pp = _step8_ptrs(master, moments8, scales8, grad, gd, param_out, n, dev)
    _L.check(_L.lib().zero_shard_adam8_step(pm, pc, ps, pg, gd, pp, pd, n, ctypes.byref(params), _seed(seed),
                                            _buf(global_sqnorm, torch.float64, 8, "global_sqnorm", dev),
                                            _buf(global_overflow, torch.int32, 4, "global_overflow", dev), _stream(stream, dev)),
             "zero_shard_adam8_step")


def zero_shard_adam8_step_coef(master, moments8, scales8, grad, param_out, d_coef, d_step, global_sqnorm,
                               global_overflow=None, seed: int = 0, grad_dtype: Optional[int] = None,
                               param_dtype: Optional[int] = None, n: Optional[int] = None, stream=None) -> None:
    """zero_shard_adam8_step with the coefficient block read from device memory
    d_coef and the step that keys the rounding from d_step (int64 [1])."""
    gd = dtype_code(grad if grad_dtype is None else grad_dtype)
    pd = 0 if param_out is None else dtype_code(param_out if param_dtype is None else param_dtype)
    n = master.numel() if n is None else n
    dev = _current_device()
    pm, pc, ps, pg, pp = _step8_ptrs(master, moments8, scales8, grad, gd, param_out, n, dev)
    _L.check(_L.lib().zero_shard_adam8_step_coef(pm, pc, ps, pg, gd, pp, pd, n, _buf(d_coef, None, zero_adam_coef_bytes(), "d_coef", dev),
                                                 _seed(seed),
                                                 _buf(d_step, torch.int64, 8, "d_step", dev),
                                                 _buf(global_sqnorm, torch.float64, 8, "global_sqnorm", dev),
                                                 _buf(global_overflow, torch.int32, 4, "global_overflow", dev),
                                                 _stream(stream, dev)), "zero_shard_adam8_step_coef")


def zero_moments8_pack(moments8, scales8, exp_avg, exp_avg_sq, n: Optional[int] = None, stream=None) -> None:
    """Codes and block scales of fp32 moments, rounded to nearest."""
    n = exp_avg.numel() if n is None else n
    dev = _current_device()
    _L.check(_L.lib().zero_moments8_pack(_buf(moments8, torch.uint8, _codes_bytes(n), "moments8", dev),
                                         _buf(scales8, torch.uint8, _scales_bytes(n), "scales8", dev),
                                         _buf(exp_avg, torch.float32, 4 * n, "exp_avg", dev), _buf(exp_avg_sq, torch.float32, 4 * n, "exp_avg_sq", dev), n,
                                         _stream(stream, dev)), "zero_moments8_pack")


def zero_moments8_unpack(exp_avg, exp_avg_sq, moments8, scales8, n: Optional[int] = None, stream=None) -> None:
    """fp32 moments from their codes and block scales."""
    n = exp_avg.numel() if n is None else n
    dev = _current_device()
    _L.check(_L.lib().zero_moments8_unpack(_buf(exp_avg, torch.float32, 4 * n, "exp_avg", dev), _buf(exp_avg_sq, torch.float32, 4 * n, "exp_avg_sq", dev),
                                           _buf(moments8, torch.uint8, _codes_bytes(n), "moments8", dev),
                                           _buf(scales8, torch.uint8, _scales_bytes(n), "scales8", dev), n, _stream(stream, dev)),
             "zero_moments8_unpack")
