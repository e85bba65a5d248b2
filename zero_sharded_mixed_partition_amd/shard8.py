"""ShardAdam8: ShardAdam with its moments in 8 bits, 2.06 bytes a parameter
instead of 8 (the format: include/zero_shard.h).  The norm pass, accumulation,
reduction, loss scaling and the device-resident step state are ShardAdam's;
only the update differs."""
from typing import Optional

import torch

from . import ZERO_F32, AdamHyper, LossScaler, dtype_code
from .moments8 import (zero_moments8_bytes, zero_moments8_pack, zero_moments8_unpack, zero_scales8_bytes,
                       zero_shard_adam8_step, zero_shard_adam8_step_coef)
from .shard import ShardAdam


class ShardAdam8(ShardAdam):
    def __init__(self, master: torch.Tensor, moments8: Optional[torch.Tensor] = None,
                 scales8: Optional[torch.Tensor] = None, *, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8,
                 weight_decay=0.0, max_grad_norm=0.0, scaler: Optional[LossScaler] = None, applied_steps: int = 0,
                 device_state: bool = False, seed: int = 0):
        """moments8, scales8: uint8 device tensors of zero_moments8_bytes(n) and
        zero_scales8_bytes(n) bytes, or None for moments of zero.  seed keys the
        stochastic rounding (with the step's and the element's index), so equal
        runs agree bit for bit; give each rank its own, else their shards are
        rounded with the same words.  A step with device_state=True can be recorded
        in a torch CUDA graph, which keeps the hyperparameters and the seed of its
        recording."""
        if master.dtype != torch.float32 or not master.is_cuda or not master.is_contiguous():
            raise ValueError("master must be a contiguous fp32 device tensor")
        if (moments8 is None) != (scales8 is None):
            raise ValueError("moments8 and scales8 belong together")
        n = master.numel()
        sizes = zero_moments8_bytes(n), zero_scales8_bytes(n)
        if moments8 is None:
            moments8, scales8 = (torch.zeros(k, dtype=torch.uint8, device=master.device) for k in sizes)
        for t, k in zip((moments8, scales8), sizes):
            if t.dtype != torch.uint8 or not t.is_cuda or t.numel() != k or not t.is_contiguous():
                raise ValueError(f"moments8 / scales8 must be contiguous uint8 device tensors of {sizes} bytes")
        self.master, self.moments8, self.scales8, self.seed = master, moments8, scales8, int(seed)
        self._init_step(n, dict(lr=lr, beta1=beta1, beta2=beta2, eps=eps, weight_decay=weight_decay,
                                max_grad_norm=max_grad_norm), scaler, applied_steps, False, device_state)

    @classmethod
    def from_moments(cls, master: torch.Tensor, exp_avg: torch.Tensor, exp_avg_sq: torch.Tensor, **kw) -> "ShardAdam8":
        """A shard that goes over from fp32 moments (rounded to nearest); the
        fp32 ones are no longer needed once the stream has passed this point."""
        n = master.numel()
        c, s = (torch.empty(k, dtype=torch.uint8, device=master.device)
                for k in (zero_moments8_bytes(n), zero_scales8_bytes(n)))
        zero_moments8_pack(c, s, exp_avg, exp_avg_sq, n=n)
        return cls(master, c, s, **kw)

    def moments(self):
        """(exp_avg, exp_avg_sq) as new fp32 tensors."""
        m, v = torch.empty_like(self.master), torch.empty_like(self.master)
        zero_moments8_unpack(m, v, self.moments8, self.scales8)
        return m, v

    def checkpoint_arrays(self) -> dict:
        return {"master": self.master, "moments8": self.moments8, "scales8": self.scales8}

    def apply(self, grad: torch.Tensor, param_out: Optional[torch.Tensor], global_sqnorm=None,
              global_overflow=None) -> None:
        if self.state is not None:
            super().apply(grad, param_out, global_sqnorm, global_overflow)
            return
        inv = 1.0 if dtype_code(grad) == ZERO_F32 else 1.0 / self.scaler.scale
        zero_shard_adam8_step(self.master, self.moments8, self.scales8, grad, param_out,
                              AdamHyper(step=self.t + 1, inv_loss_scale=inv, **self.hyper),
                              self.sqnorm if global_sqnorm is None else global_sqnorm,
                              self.overflow if global_overflow is None else global_overflow, seed=self.seed)

    def update(self, grad: torch.Tensor, param_out: Optional[torch.Tensor], global_sqnorm=None,
               global_overflow=None) -> None:
        # after the decision the state's applied count is the step's index (a skipped step writes nothing)
        zero_shard_adam8_step_coef(self.master, self.moments8, self.scales8, grad, param_out, self.d_coef,
                                   self.state.applied(), self.sqnorm if global_sqnorm is None else global_sqnorm,
                                   self.overflow if global_overflow is None else global_overflow, seed=self.seed)
