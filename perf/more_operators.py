"""Cases that measure the operators of a step by orthogonalised momentum over a
list of matrices: the momentum pass (unscale, clip, exponential average, Nesterov
form), the orthogonalisation of its updates by a quintic Newton-Schulz iteration,
and the update of the master weights and their 16-bit copies by the result.

`own` chooses what run() computes with: False, elementary torch operations in 32
bits on whole buffers (the matrices of one shape as one batched product), rounded
once at the end; True, the package's calls.

A list is written as text: "8x4096x4096 4x11008x4096" are eight matrices of 4096
rows and 4096 columns and four of 11008 x 4096."""
import math

import torch

own = False

_TYPE = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_MU, _LR, _DECAY, _CLIP, _EPS = 0.95, 2e-2, 0.1, 1.0, 1e-7
_COEFS = ((3.4445, -4.7750, 2.0315),) * 5
_GROWTH = 0.2                         # updates are scaled to 0.2 times an orthogonal matrix's largest side's root


# ---------------------------------------------------------------- cases

def listed():
    toy = "4x512x512 4x1024x512 2x512x1024"                         # a toy decoder: a launch costs more than the bytes
    odd = "24x331x331 12x881x331 6x331x881"                         # six layers, no side a multiple of four, end to end
    big = "8x4096x4096 4x11008x4096 2x4096x11008"                   # two layers at the widths of a 7B model
    return [
        dict(name="momentum toy fp16", op="momentum", shapes=toy, grad="f16", update="bf16", nesterov=True, packed=False),
        dict(name="momentum odd fp32 out", op="momentum", shapes=odd, grad="bf16", update="f32", nesterov=False,
             packed=True),
        dict(name="momentum 405M bf16", op="momentum", shapes=big, grad="bf16", update="bf16", nesterov=True,
             packed=False),
        # one matrix alone: the shortest chain of dependent products
        dict(name="orthogonalize one 512", op="orthogonalize", shapes="1x512x512", update="bf16", batched=False,
             packed=False),
        dict(name="orthogonalize odd", op="orthogonalize", shapes=odd, update="bf16", batched=False, packed=True),
        # low-rank adapters of 32 projections: both factors, one wide and one tall
        dict(name="orthogonalize rank 16", op="orthogonalize", shapes="32x16x4096 32x4096x16", update="f32",
             batched=False, packed=False),
        # the query and key projections of a layer, head by head
        dict(name="orthogonalize heads", op="orthogonalize", shapes="64x128x4096", update="f16", batched=True,
             packed=False),
        # a layer of 32 experts: gate, up and down projections
        dict(name="orthogonalize experts", op="orthogonalize", shapes="64x1408x2048 32x2048x1408", update="bf16",
             batched=True, packed=False),
        dict(name="orthogonalize 405M", op="orthogonalize", shapes=big, update="bf16", batched=False, packed=False),
        dict(name="update toy", op="update", shapes=toy, param="f16", packed=False),
        dict(name="update odd no copy", op="update", shapes=odd, param="none", packed=True),
        dict(name="update 405M bf16", op="update", shapes=big, param="bf16", packed=False),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["momentum", "orthogonalize", "orthogonalize", "update"])
    while True:
        groups = [(log(1, 48), log(16, 11008), log(16, 11008)) for _ in range(rng.randint(1, 3))]
        if sum(k * r * c for k, r, c in groups) > 200_000_000 or sum(k for k, _, _ in groups) > 100:
            continue
        case = dict(op=op, shapes=" ".join("%dx%dx%d" % g for g in groups), packed=rng.random() < 0.5)
        if op == "orthogonalize" and work(dict(case, update="f32"))["flops"] > 3e12:
            continue
        if op == "update":
            return dict(case, param=rng.choice(["f16", "bf16", "none"]))
        case["update"] = rng.choice(["bf16", "bf16", "f16", "f32"] if op == "orthogonalize" else ["bf16", "f32"])
        if op == "orthogonalize":
            return dict(case, batched=rng.random() < 0.3)
        return dict(case, grad=rng.choice(["f16", "bf16", "f32"]), nesterov=rng.random() < 0.7)


def _groups(case):
    """(matrices, rows, columns) of each group of matrices of one shape."""
    return [tuple(int(x) for x in part.split("x")) for part in case["shapes"].split()]


def _layout(case):
    """Where each group starts in a flat buffer, and the buffer's length.  packed:
    end to end; else every group starts at a multiple of 32 elements."""
    starts, at, step = [], 0, 1 if case["packed"] else 32
    for k, r, c in _groups(case):
        starts.append(at)
        at += -(-k * r * c // step) * step
    return starts, at


def work(case):
    n = sum(k * r * c for k, r, c in _groups(case))
    if case["op"] == "momentum":
        out = 4 if case["update"] == "f32" else 2
        return {"bytes": n * ((4 if case["grad"] == "f32" else 2) + 8 + out), "flops": 6 * n}
    if case["op"] == "update":
        return {"bytes": n * (10 + (0 if case["param"] == "none" else 2)), "flops": 2 * n}
    # For sides s <= l: a symmetric product costs half of a general one.  Either the
    # iteration as it stands, per step X X^T (s s l), its square (s s s) and the
    # product with X (2 s s l); or all of it in the symmetric s x s matrices
    # (17 s s s) between one X X^T and one product with X.
    flops = 0
    for k, r, c in _groups(case):
        s, l = min(r, c), max(r, c)
        flops += k * min(len(_COEFS) * (3 * s * s * l + s ** 3), 3 * s * s * l + 17 * s ** 3)
    return {"bytes": n * ((4 if case["update"] == "f32" else 2) + 2), "flops": flops}


def _inv_scale(case):
    return 1.0 / 1024.0 if case.get("grad") == "f16" else 1.0


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    starts, total = _layout(case)
    op = case["op"]
    s = {"case": case, "groups": _groups(case), "starts": starts}

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def zeros(kind):
        return torch.zeros(total, dtype=_TYPE[kind], device="cuda")

    if op == "momentum":
        # elements of one matrix differ in size by a factor of some tens, as gradients do
        spread = normal(total).mul_(0.8).exp_().mul_(1e-3)
        s["grad"] = normal(total).mul_(spread).div_(_inv_scale(case)).to(_TYPE[case["grad"]])
        s["momentum"] = normal(total).mul_(spread).mul_(0.3)
        s["update"] = zeros(case["update"])
        s["global_sqnorm"] = torch.full((1,), 4.0, dtype=torch.float64, device="cuda")
    elif op == "orthogonalize":
        # momentum of a training run: a few strong directions over noise, rows and columns of different size
        u = torch.empty(total, device="cuda")
        for (k, r, c), a in zip(s["groups"], starts):
            rank = max(1, min(r, c) // 16)
            x = torch.matmul(normal(k, r, rank) * torch.linspace(0.0, -2.0, rank, device="cuda").exp(), normal(k, rank, c))
            x = x.mul_(0.7 / math.sqrt(rank)).add_(normal(k, r, c))
            x *= normal(k, r, 1).mul_(0.3).exp_() * normal(k, 1, c).mul_(0.3).exp_()
            u[a:a + k * r * c] = x.mul_(1e-3).view(-1)
            del x
        s["update"] = u.to(_TYPE[case["update"]])
        s["ortho"] = zeros("bf16")
    else:
        s["master"] = normal(total).mul_(0.02)
        s["ortho"] = torch.empty(total, dtype=torch.bfloat16, device="cuda")
        for (k, r, c), a in zip(s["groups"], starts):
            s["ortho"][a:a + k * r * c] = normal(k * r * c).div_(math.sqrt(max(r, c)))
        s["param"] = None if case["param"] == "none" else zeros(case["param"])
    if own:
        import zero_sharded_mixed_partition_amd as Z

        # what lies between two groups is updated with the buffer it is in, as a row of its own
        ends = [a + k * r * c for (k, r, c), a in zip(s["groups"], starts)]
        gaps = [(a, b) for a, b in zip(ends, starts[1:] + [total]) if a < b and op != "orthogonalize"]
        if op == "update":
            for a, b in gaps:
                s["ortho"][a:b] = 0.0

        def views(flat):
            if flat is None:
                return None
            three = [flat[a:a + k * r * c].view(k, r, c) for (k, r, c), a in zip(s["groups"], starts)]
            return (three if case.get("batched") else [x for g in three for x in g]) + [flat[a:b].view(1, -1) for a, b in gaps]

        lists = {"momentums": views(s.get("momentum")), "grads": views(s.get("grad")), "masters": views(s.get("master")),
                 "params_out": views(s.get("param")), "updates": views(s.get("update")), "orthos": views(s.get("ortho"))}
        if op == "update":
            lists["scales"] = [_growth(k, r, c) for k, r, c in s["groups"] for _ in range(k)] + [0.0] * len(gaps)
        s["table"] = Z.MatrixTable(**{k: v for k, v in lists.items() if v is not None})
        if op == "orthogonalize":
            s["workspace"] = torch.empty(Z.zero_multi_orthogonalize_workspace_bytes(s["table"]), dtype=torch.uint8,
                                         device="cuda")
    return s


def _growth(k, r, c):
    return _GROWTH * math.sqrt(max(r, c))


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        _run_own(s)
    elif op == "momentum":
        _plain_momentum(s)
    elif op == "orthogonalize":
        _plain_orthogonalize(s)
    else:
        _plain_update(s)
    names = {"momentum": ("momentum", "update"), "orthogonalize": ("ortho",), "update": ("master", "param")}[op]
    return {k: s[k] for k in names}


def _run_own(s):
    import zero_sharded_mixed_partition_amd as Z
    case = s["case"]
    if case["op"] == "orthogonalize":
        Z.zero_multi_orthogonalize(s["table"], s["workspace"], coefs=_COEFS, eps=_EPS)
        return
    hp = [Z.MuonHyper(lr=_LR, momentum=_MU, weight_decay=_DECAY, nesterov=case.get("nesterov", True))]
    if case["op"] == "momentum":
        Z.zero_multi_momentum_step(s["table"], hp, inv_loss_scale=_inv_scale(case), max_grad_norm=_CLIP,
                                   global_sqnorm=s["global_sqnorm"])
    else:
        Z.zero_multi_muon_update(s["table"], hp)


# ---------------------------------------------------------------- plain forms

def _plain_momentum(s):
    clip = (_CLIP / (s["global_sqnorm"].sqrt() + 1e-6)).clamp(max=1.0) * _inv_scale(s["case"])
    g = s["grad"].float() * (clip.float() * (1 - _MU))
    m = s["momentum"].mul_(_MU).add_(g)
    s["update"].copy_(m * _MU + g if s["case"]["nesterov"] else m)


def _plain_orthogonalize(s):
    for (k, r, c), a in zip(s["groups"], s["starts"]):
        x = s["update"][a:a + k * r * c].view(k, r, c).float()
        if r > c:
            x = x.transpose(1, 2).contiguous()
        norm = x.square().sum((1, 2), keepdim=True, dtype=torch.float64).sqrt().clamp(min=_EPS)
        x = x / norm.float()
        for p, q, t in _COEFS:
            gram = torch.matmul(x, x.transpose(1, 2))
            x = x * p + torch.matmul(gram * q + torch.matmul(gram, gram) * t, x)
        s["ortho"][a:a + k * r * c].view(k, r, c).copy_(x.transpose(1, 2) if r > c else x)


def _plain_update(s):
    keep = 1 - _LR * _DECAY
    p = s["master"].mul_(keep)
    for (k, r, c), a in zip(s["groups"], s["starts"]):
        p[a:a + k * r * c] -= s["ortho"][a:a + k * r * c].float() * (_LR * _growth(k, r, c))
    if s["param"] is not None:
        s["param"].copy_(p)


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "momentum":
        coef = min(1.0, _CLIP / (math.sqrt(float(s["global_sqnorm"])) + 1e-6)) * _inv_scale(case)
        g = s["grad"].to(torch.float64) * coef
        m = _MU * s["momentum"].to(torch.float64) + (1 - _MU) * g
        return {"momentum": m, "update": (1 - _MU) * g + _MU * m if case["nesterov"] else m}
    if case["op"] == "update":
        p = s["master"].to(torch.float64)
        for (k, r, c), a in zip(s["groups"], s["starts"]):
            z = slice(a, a + k * r * c)
            p[z] = p[z] - _LR * (_DECAY * p[z] + _GROWTH * max(r, c) ** 0.5 * s["ortho"][z].to(torch.float64))
        return {"master": p, "param": None if s["param"] is None else p}
    out = torch.zeros(s["update"].numel(), dtype=torch.float64, device="cuda")
    for (k, r, c), a in zip(s["groups"], s["starts"]):
        for i in range(k):
            z = slice(a + i * r * c, a + (i + 1) * r * c)
            x = s["update"][z].to(torch.float64).view(r, c)
            x = x / max(float(torch.linalg.matrix_norm(x)), _EPS)
            for p, q, t in _COEFS:                                  # p x + q (x x^T) x + t (x x^T)^2 x, from the left or right
                if r <= c:
                    w = x @ x.t()
                    y = w @ x
                    x = p * x + q * y + t * (w @ y)
                else:
                    w = x.t() @ x
                    y = x @ w
                    x = p * x + q * y + t * (y @ w)
            out[z] = x.reshape(-1)
    return {"ortho": out}
