"""Checkpoint and resume of one rank's optimizer shard.

The shard state is the checkpoint unit of a ZeRO rank: its fp32 master,
exp_avg and exp_avg_sq partitions plus the step scalars (applied steps, loss
scaler).  save() writes them as one .npy file each and one JSON file in a
directory; load() restores them into a ShardAdam built over the same shard
size.  ShardAdam8 saves its 8-bit moments as they are (codes and scales), and
the seed of their rounding; MultiAdam saves its tensors in list order, and the
group of each: a list of other tensors or with other groups is refused.  MultiMuon
also saves what its steps are made of besides the hyperparameters (coefs, eps, each
matrix's factor of the learning rate, the type of its updates): others are refused.
Because every step is deterministic, k steps, save, load and k more steps give the same
bits as 2k uninterrupted steps.
"""
import copy
import json
import os

import numpy as np
import torch

_SCALER = ("scale", "min_scale", "backoff", "growth", "growth_interval", "good_steps")


def state_dict(opt) -> dict:
    """Host copies of the shard and its scalars (waits for queued steps)."""
    skipped = 0
    if opt.state is not None:
        skipped = opt.read_state().skipped          # refreshes opt.t and opt.scaler
    torch.cuda.current_stream().synchronize()
    d = {k: x.cpu().numpy() for k, x in opt.checkpoint_arrays().items()}
    d["t"] = int(opt.t)
    d["skipped"] = int(skipped)
    d["scaler"] = {k: getattr(opt.scaler.s, k) for k in _SCALER}
    d["hyper"] = copy.deepcopy(opt.hyper)
    if hasattr(opt, "seed"):
        d["seed"] = opt.seed                           # keys the rounding of 8-bit moments
    if hasattr(opt, "groups"):
        d["groups"] = list(opt.groups)                 # one per tensor of a list
    if hasattr(opt, "checkpoint_settings"):
        d["settings"] = opt.checkpoint_settings()
    return d


def load_state_dict(opt, d: dict) -> None:
    """Restore a state_dict into opt (same shard size and dtypes)."""
    from . import LossScaler, StepState
    arrays = opt.checkpoint_arrays()
    for k, dst in arrays.items():
        if k not in d:
            raise ValueError(f"{k}: not in the checkpoint")
        src, want = np.asarray(d[k]), str(dst.dtype).replace("torch.", "")
        if src.dtype.name != want or src.shape not in ((dst.numel(),), tuple(dst.shape)):
            raise ValueError(f"{k}: expected {want}{list(dst.shape)}, got {src.dtype}{list(src.shape)}")
    if isinstance(opt.hyper, list) and len(d["hyper"]) != len(opt.hyper):
        raise ValueError(f"{len(d['hyper'])} groups in the checkpoint, {len(opt.hyper)} expected")
    have, want = d.get("groups"), list(getattr(opt, "groups", ()))
    if have is not None and list(have) != want:
        raise ValueError(f"{len(have)} tensors in the checkpoint, {len(want)} expected" if len(have) != len(want) else
                         "the checkpoint's tensors belong to other groups")
    if d.get("settings") is not None:
        mine = opt.checkpoint_settings() if hasattr(opt, "checkpoint_settings") else {}
        for k, x in d["settings"].items():
            if mine.get(k) != x:
                raise ValueError(f"the checkpoint was written with other {k}: {x}, not {mine.get(k)}")
    for k, dst in arrays.items():
        dst.copy_(torch.from_numpy(np.ascontiguousarray(d[k])).view(dst.shape))
    opt.t = int(d["t"])
    opt.scaler = LossScaler(**d["scaler"])
    opt.hyper = copy.deepcopy(d["hyper"])
    if "seed" in d:
        opt.seed = int(d["seed"])
    if opt.state is not None:
        # in place: a step recorded in a graph keeps reading this state
        dev = opt.state.tensor.device
        fresh = StepState(opt.scaler, opt.t, dev)
        if d.get("skipped"):
            st = fresh.read()
            st.skipped = int(d["skipped"])
            fresh.tensor.copy_(torch.frombuffer(bytearray(bytes(st)), dtype=torch.uint8))
        opt.state.tensor.copy_(fresh.tensor)
    opt._graph, opt._graph_key = None, None          # a recorded step holds its hyperparameters
    torch.cuda.current_stream().synchronize()


def save(opt, directory: str) -> None:
    os.makedirs(directory, exist_ok=True)
    d = state_dict(opt)
    for k in opt.checkpoint_arrays():
        np.save(os.path.join(directory, f"{k}.npy"), d[k])
    meta = {k: d[k] for k in ("t", "skipped", "scaler", "hyper", "seed", "groups", "settings") if k in d}
    with open(os.path.join(directory, "scalars.json"), "w") as f:
        json.dump(meta, f, indent=1)


def load(opt, directory: str) -> None:
    d = {k: np.load(os.path.join(directory, f"{k}.npy"), allow_pickle=False) for k in opt.checkpoint_arrays()}
    with open(os.path.join(directory, "scalars.json")) as f:
        d.update(json.load(f))
    load_state_dict(opt, d)
