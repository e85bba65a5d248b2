"""Cases that measure the optimizer operators on lists of tensors and on 8-bit
moments: the norm pass over a list of gradients, AdamW over a list of tensors
with 32-bit and with 8-bit moments, AdamW over one flat shard with 8-bit
moments, and the conversion of moments between 32 and 8 bits.

`own` chooses what run() computes with: False, elementary torch operations on
the whole buffers; True, the package's calls.  Every operation of an update is
rounded to float32 where the kernels round it (formed in float64 first, where
a fused multiply-add or a value next to a rounding border needs it).

8-bit moments: a tensor's elements form blocks of 32.  exp_avg and the square
root of exp_avg_sq are each held as e4m3 numbers times a power of two per
block.  Codes lie in quads, four of exp_avg then four of the root, and the
two exponent bytes of a block side by side.  run() returns the codes and the
block scales as the numbers they are (float8_e4m3fn, float8_e8m0fnu); a moment
is their product."""
import math

import torch

own = False

_GRAD = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_LR, _B1, _B2, _EPS, _STEP, _CLIP = 1e-3, 0.9, 0.999, 1e-8, 100, 1.0
_DECAY = (0.1, 0.0)                   # weight decay of matrices, and of norms' vectors


# ---------------------------------------------------------------- cases

def listed():
    big = dict(vocab=32000, width=4096, ffn=11008, layers=4)        # four layers at the widths of a 7B model
    small = dict(vocab=512, width=512, ffn=1024, layers=1)          # where a launch costs more than the bytes
    odd = dict(vocab=5003, width=331, ffn=881, layers=6)            # no tensor a multiple of four, none aligned
    return [
        dict(name="norm small fp16", op="norm", grad="f16", packed=False, **small),
        dict(name="norm 1.1B bf16", op="norm", grad="bf16", packed=False, **big),
        dict(name="adam list odd packed bf16", op="adam", grad="bf16", param="bf16", packed=True, **odd),
        dict(name="adam list 1.1B bf16", op="adam", grad="bf16", param="bf16", packed=False, **big),
        dict(name="adam8 list small fp32 grad", op="adam8", grad="f32", param="bf16", packed=False, **small),
        dict(name="adam8 list 1.1B bf16", op="adam8", grad="bf16", param="bf16", packed=False, **big),
        # one rank's shard: a toy model's quarter, and one of 400 ranks of a 100B model
        dict(name="shard8 197k fp16", op="shard8", grad="f16", param="f16", n=196864),
        dict(name="shard8 251M fp16", op="shard8", grad="f16", param="f16", n=250749440),
        # a run that goes over to 8-bit moments, and one that reads them back (a checkpoint)
        dict(name="pack 15.6M", op="pack", n=15555077),
        dict(name="pack 251M", op="pack", n=250749440),
        dict(name="unpack 1M odd", op="unpack", n=1000003),
        dict(name="unpack 251M", op="unpack", n=250749440),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "adam", "adam8", "shard8", "pack", "unpack"])
    if op in ("pack", "unpack"):
        return dict(op=op, n=log(1000, 250_000_000))
    case = dict(op=op, grad=rng.choice(["f16", "bf16", "f32"]))
    if op != "norm":
        case["param"] = rng.choice(["f16", "bf16", "none"])
    if op == "shard8":
        return dict(case, n=log(1000, 250_000_000))
    while True:
        model = dict(vocab=log(64, 50257), width=log(24, 4096), layers=rng.randint(0, 8))
        model["ffn"] = int(model["width"] * rng.uniform(2.0, 3.5))
        if sum(a * b for a, b in _shapes(model)) <= 600_000_000:
            return dict(case, packed=op != "adam8" and rng.random() < 0.5, **model)


def _shapes(case):
    """(rows, columns) of a decoder's tensors, in order; a vector has one row."""
    d, f = case["width"], case["ffn"]
    layer = [(1, d), (d, d), (d, d), (d, d), (d, d), (1, d), (f, d), (f, d), (d, f)]
    return [(case["vocab"], d)] + layer * case["layers"] + [(1, d), (case["vocab"], d)]


def _layout(case):
    """Starts, sizes and groups of the tensors in their flat buffers, and the
    buffers' length.  packed: end to end; else every tensor starts at a
    multiple of 32 elements, as separate allocations are aligned."""
    if "n" in case:
        return [0], [case["n"]], [0], case["n"]
    step = 1 if case["packed"] else 32
    starts, sizes, groups, at = [], [], [], 0
    for rows, cols in _shapes(case):
        starts.append(at)
        sizes.append(rows * cols)
        groups.append(1 if rows == 1 else 0)
        at += -(-rows * cols // step) * step
    return starts, sizes, groups, at


def work(case):
    _, sizes, _, _ = _layout(case)
    n, op = sum(sizes), case["op"]
    if op in ("pack", "unpack"):
        return {"bytes": n * (8 + 2 + 2 / 32), "flops": n * 6}
    g = 4 if case["grad"] == "f32" else 2
    if op == "norm":
        return {"bytes": n * g + 8 * len(sizes), "flops": n * 2}
    p = 0 if case["param"] == "none" else 2
    moments = 16 if op == "adam" else 4 + 4 / 32
    return {"bytes": n * (g + p + 8 + moments), "flops": n * 20}


def _inv_scale(case):
    return 1.0 / 1024.0 if case["grad"] == "f16" else 1.0


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    starts, sizes, groups, total = _layout(case)
    op = case["op"]
    s = {"case": case, "starts": starts, "sizes": sizes, "groups": groups, "seed": seed}

    def normal():
        return torch.randn(total, generator=gen, device="cuda")

    # elements of one tensor differ in size by a factor of some tens, as gradients do
    spread = normal().mul_(0.8).exp_().mul_(1e-3)
    gaps = None
    if total != sum(sizes):                                       # zeros between the tensors, in every buffer
        gaps = torch.ones(total, dtype=torch.bool, device="cuda")
        for a, b in zip(starts, sizes):
            gaps[a:a + b] = False
        spread.masked_fill_(gaps, 0.0)
    if op not in ("pack", "unpack"):
        s["grad"] = normal().mul_(spread).div_(_inv_scale(case)).to(_GRAD[case["grad"]])
    if op == "norm":
        s["sqnorm"] = torch.empty(1, dtype=torch.float64, device="cuda")
        s["overflow"] = torch.empty(1, dtype=torch.int32, device="cuda")
        s["tensor_sqnorm"] = torch.empty(len(sizes), dtype=torch.float64, device="cuda")
    else:
        exp_avg = normal().mul_(spread).mul_(0.3)
        exp_avg_sq = torch.rand(total, generator=gen, device="cuda").add_(0.5).mul_(spread.square_())
        del spread
        if op in ("adam", "pack"):
            s["exp_avg"], s["exp_avg_sq"] = exp_avg, exp_avg_sq
        if op == "pack":
            s["moments8"] = torch.zeros(8 * -(-total // 4), dtype=torch.uint8, device="cuda")
            s["scales8"] = torch.zeros(2 * -(-total // 32), dtype=torch.uint8, device="cuda")
        elif op != "adam":
            s["moments8"], s["scales8"] = _codes(exp_avg, exp_avg_sq.sqrt_(), None)
        if op == "unpack":
            s["exp_avg"], s["exp_avg_sq"] = torch.empty_like(exp_avg), torch.empty_like(exp_avg)
    if op in ("adam", "adam8", "shard8"):
        s["master"] = normal().mul_(0.02)
        if gaps is not None:
            s["master"].masked_fill_(gaps, 0.0)
        s["param"] = None if case["param"] == "none" else torch.zeros(total, dtype=_GRAD[case["param"]], device="cuda")
        s["global_sqnorm"] = torch.full((1,), 4.0, dtype=torch.float64, device="cuda")
        s["global_overflow"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if own:
        import zero_sharded_mixed_partition_amd as Z

        def views(flat):
            return [flat[a:a + b] for a, b in zip(starts, sizes)]

        if op == "norm":
            s["table"] = Z.TensorTable.of_grads(views(s["grad"]))
            s["workspace"] = torch.empty(Z.zero_multi_norm_workspace_bytes(s["table"]), dtype=torch.uint8,
                                         device="cuda")
        elif op in ("adam", "adam8"):
            out = None if s["param"] is None else views(s["param"])
            if op == "adam":
                moments = views(s["exp_avg"]), views(s["exp_avg_sq"])
            else:
                moments = ([s["moments8"][2 * a:2 * a + 8 * -(-b // 4)] for a, b in zip(starts, sizes)],
                           [s["scales8"][a // 16:a // 16 + 2 * -(-b // 32)] for a, b in zip(starts, sizes)])
            s["table"] = Z.TensorTable(views(s["master"]), *moments, views(s["grad"]), out, groups=groups,
                                       state_bits=32 if op == "adam" else 8)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        _run_own(s)
    elif op == "norm":
        _plain_norm(s)
    elif op == "pack":
        s["moments8"], s["scales8"] = _codes(s["exp_avg"], s["exp_avg_sq"].sqrt(), None)
    elif op == "unpack":
        _plain_unpack(s)
    else:
        _plain_adam(s)
    if op == "norm":
        return {k: s[k] for k in ("sqnorm", "overflow", "tensor_sqnorm")}
    if op == "unpack":
        return {k: s[k] for k in ("exp_avg", "exp_avg_sq")}
    out = {} if op == "pack" else {"master": s["master"], "param": s["param"]}
    if op == "adam":
        return dict(out, exp_avg=s["exp_avg"], exp_avg_sq=s["exp_avg_sq"])
    return dict(out, codes=s["moments8"].view(torch.float8_e4m3fn), scales=s["scales8"].view(torch.float8_e8m0fnu))


def _run_own(s):
    import zero_sharded_mixed_partition_amd as Z
    case = s["case"]
    op = case["op"]
    if op == "norm":
        Z.zero_multi_unscale_norm_overflow(s["table"], _inv_scale(case), s["sqnorm"], s["overflow"], s["workspace"],
                                           s["tensor_sqnorm"])
        return
    if op == "pack":
        Z.zero_moments8_pack(s["moments8"], s["scales8"], s["exp_avg"], s["exp_avg_sq"])
        return
    if op == "unpack":
        Z.zero_moments8_unpack(s["exp_avg"], s["exp_avg_sq"], s["moments8"], s["scales8"])
        return
    hp = [Z.AdamHyper(lr=_LR, beta1=_B1, beta2=_B2, eps=_EPS, weight_decay=wd, step=_STEP,
                      inv_loss_scale=_inv_scale(case), max_grad_norm=_CLIP) for wd in _DECAY]
    if op == "shard8":
        Z.zero_shard_adam8_step(s["master"], s["moments8"], s["scales8"], s["grad"], s["param"], hp[0],
                                s["global_sqnorm"], s["global_overflow"], seed=s["seed"])
    else:
        Z.zero_multi_adam_step(s["table"], hp, s["global_sqnorm"], s["global_overflow"], seed=s["seed"])


# ---------------------------------------------------------------- plain forms

def _plain_norm(s):
    g = s["grad"]
    sums = torch.stack([g[a:a + b].double().square().sum() for a, b in zip(s["starts"], s["sizes"])])
    s["tensor_sqnorm"] = sums * _inv_scale(s["case"]) ** 2
    s["sqnorm"] = s["tensor_sqnorm"].sum().reshape(1)
    s["overflow"] = (~torch.isfinite(g).all()).int().reshape(1)


def _f32(x):
    return x.float().double()


def _lengths(s):
    """Elements from each tensor's start to the next one's."""
    return [b - a for a, b in zip(s["starts"], s["starts"][1:] + [s["grad"].numel()])]


def _per_element(s, values):
    """One float32 value per element from one per group."""
    return torch.cat([torch.full((n,), values[k], device="cuda") for n, k in zip(_lengths(s), s["groups"])])


def _plain_adam(s):
    """Master, moments and the 16-bit copy, each operation rounded to float32."""
    case = s["case"]
    c = {k: float(torch.tensor(v, dtype=torch.float32)) for k, v in dict(
        b1=_B1, o1=1 - _B1, b2=_B2, o2=1 - _B2, ss=_LR / (1 - _B1 ** _STEP), rb=1 / math.sqrt(1 - _B2 ** _STEP),
        eps=_EPS).items()}
    n, eight = s["master"].numel(), case["op"] != "adam"
    clip = (_CLIP / (s["global_sqnorm"].sqrt() + 1e-6)).clamp(max=1.0)
    g = _f32(s["grad"].double() * (clip * _inv_scale(case)).float())
    if eight:
        m, root = _moments(s["moments8"], s["scales8"], n)
        m, v = m.double(), _f32(root.double().square())
        del root
    else:
        m, v = s["exp_avg"].double(), s["exp_avg_sq"].double()
    m = _f32(c["b1"] * m + _f32(c["o1"] * g))
    v = _f32(c["b2"] * v + _f32(_f32(c["o2"] * g) * g))
    del g
    root = _f32(v.sqrt())
    u = _f32(_f32(c["ss"] * m) / _f32(root * c["rb"] + c["eps"]))
    p = (s["master"].double() * _per_element(s, [1 - _LR * wd for wd in _DECAY]) - u).float()
    del u
    s["master"].copy_(p)
    if s["param"] is not None:
        s["param"].copy_(p)
    if not eight:
        s["exp_avg"].copy_(m)
        s["exp_avg_sq"].copy_(v)
        return
    codes, scales = _codes(m.float(), root.float(), _random(s))
    s["moments8"].copy_(codes)
    s["scales8"].copy_(scales)


def _plain_unpack(s):
    m, root = _moments(s["moments8"], s["scales8"], s["exp_avg"].numel())
    s["exp_avg"].copy_(m)
    s["exp_avg_sq"].copy_(root.square())


def _power(byte):
    """2 ** (byte - 127), float32."""
    return (byte.int() << 23).view(torch.float32)


def _moments(codes, scales, n):
    """exp_avg and the root of exp_avg_sq, float32, from their codes."""
    values = codes.view(torch.float8_e4m3fn).float().view(-1, 2, 4).permute(1, 0, 2).reshape(2, -1)
    scale = _power(scales.view(-1, 2)).t().repeat_interleave(32, dim=1)[:, :values.shape[1]]
    both = values * scale
    return both[0, :n], both[1, :n]


def _random(s):
    """Two 32-bit random words per element, from the seed, the step, the
    tensor and the element's place in it."""
    mask = (1 << 64) - 1
    key = (s["seed"] * 0x9E3779B97F4A7C15 + _STEP * 0xBB67AE8584CAA73B) & mask
    key ^= key >> 32
    key = key * 0x6A09E667F3BCC909 & mask
    key = (key ^ key >> 32) & 0xFFFFFFFF
    x = torch.cat([torch.arange(n, device="cuda") ^ (key + 0x3C6EF373 * i & 0xFFFFFFFF)
                   for i, n in enumerate(_lengths(s))])
    x ^= x >> 16
    x = x * 0x9E3779B9 & 0xFFFFFFFF
    x ^= x >> 13
    x = x * 0xBB67AE85 & 0xFFFFFFFF
    x ^= x >> 16
    return x, (x << 16 | x >> 16) & 0xFFFFFFFF


def _codes(m, root, random):
    """Codes and exponent bytes of two float32 moments.  The block's largest
    magnitude lands in [128, 256); a positive root is at least the smallest
    code.  random: a word for each value, whose upper 20 bits are added below
    the last place before truncation; None rounds to nearest even."""
    n = m.numel()
    rows = -(-n // 32) * 32
    halves, scales = [], []
    for k, x in enumerate((m, root)):
        x = torch.nn.functional.pad(x, (0, rows - n)).view(-1, 32)
        byte = (x.abs().view(torch.int32) >> 23).amax(1, keepdim=True).clamp(min=8) - 7
        scale = _power(byte)
        if k == 1:
            x = torch.where(x > 0, torch.maximum(x, scale * 2.0 ** -9), x)
        y = (x.double() / scale).view(-1)
        if random is not None:
            quantum = torch.ldexp(torch.ones((), device=y.device, dtype=torch.float64),
                                  (torch.frexp(y)[1] - 1).clamp_(min=-6) - 3)
            up = torch.nn.functional.pad(random[k] >> 12, (0, rows - n)).double() / 2.0 ** 20
            y = torch.copysign((y.abs() / quantum + up).floor() * quantum, y)
        halves.append(y.float().to(torch.float8_e4m3fn).view(torch.uint8).view(-1, 4))
        scales.append(byte.to(torch.uint8))
    codes = torch.stack(halves, 1).view(-1)[:8 * -(-n // 4)]
    return codes.contiguous(), torch.cat(scales, 1).view(-1)


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        per = [(s["grad"][a:a + b].to(torch.float64) * _inv_scale(case)).pow(2).sum().item()
               for a, b in zip(s["starts"], s["sizes"])]
        return {"sqnorm": torch.tensor([math.fsum(per)], dtype=torch.float64), "overflow": None,
                "tensor_sqnorm": torch.tensor(per, dtype=torch.float64)}
    n = sum(s["sizes"]) if "n" in case else s.get("grad", s.get("exp_avg")).numel()
    out = {}
    if op in ("unpack", "adam8", "shard8"):
        value, power = _exact_tables(s["moments8"].device)
        which = torch.arange(n, device="cuda")
        at = which // 4 * 8 + which % 4
        m = value[s["moments8"][at].int()] * power[s["scales8"][which // 32 * 2].int()]
        root = value[s["moments8"][at + 4].int()] * power[s["scales8"][which // 32 * 2 + 1].int()]
        v = root * root
        del root, at, which
    else:
        m, v = s["exp_avg"].to(torch.float64), s["exp_avg_sq"].to(torch.float64)
    if op == "unpack":
        return {"exp_avg": m, "exp_avg_sq": v}
    if op != "pack":
        coef = min(1.0, _CLIP / (math.sqrt(float(s["global_sqnorm"])) + 1e-6))
        g = s["grad"].to(torch.float64) * (coef * _inv_scale(case))
        m = m * _B1 + g * (1 - _B1)
        v = v * _B2 + g.pow(2) * (1 - _B2)
        del g
        p = s["master"].to(torch.float64)
        step = (m / (1 - _B1 ** _STEP)) / ((v / (1 - _B2 ** _STEP)).sqrt() + _EPS)
        for a, b, group in zip(s["starts"], s["sizes"], s["groups"]):
            p[a:a + b] -= _LR * (step[a:a + b] + _DECAY[group] * p[a:a + b])
        del step
        out = {"master": p, "param": None if s["param"] is None else p}
        if op == "adam":
            return dict(out, exp_avg=m, exp_avg_sq=v)
    bits = None if op == "pack" else _random(s)
    codes = torch.zeros(s["moments8"].numel() // 8, 2, 4, dtype=torch.float64, device="cuda")
    scales = torch.zeros(s["scales8"].numel() // 2, 2, dtype=torch.float64, device="cuda")
    for k, x in enumerate((m, v.sqrt())):
        pad = torch.zeros(scales.shape[0] * 32, dtype=torch.float64, device="cuda")
        pad[:n] = x
        top = pad.view(-1, 32).abs().amax(1)
        e = torch.where(top > 0, torch.log2(top).floor(), torch.full_like(top, -1000.0)).clamp_(min=-119.0) - 7
        scales[:, k] = torch.exp2(e)
        y = pad.view(-1, 32) / scales[:, k:k + 1]
        if k == 1:
            y[(y > 0) & (y < 2.0 ** -9)] = 2.0 ** -9
        y = y.view(-1)[:n]
        last = torch.exp2(torch.where(y == 0, -6.0, y.abs().log2().floor().clamp_(min=-6.0)) - 3.0)
        if bits is None:
            y = torch.round(y / last) * last
        else:
            y = torch.sign(y) * torch.floor(y.abs() / last + (bits[k] >> 12) * 2.0 ** -20) * last
        pad.zero_()
        pad[:n] = y
        codes[:, k, :] = pad.view(-1, 4)[:codes.shape[0]]
    return dict(out, codes=codes.view(-1), scales=scales.view(-1))


def _exact_tables(device):
    """The value of each e4m3 code and of each exponent byte."""
    value = [(-1.0 if c & 128 else 1.0) * (math.ldexp(c & 7, -9) if not c & 120 else
                                           math.ldexp(8 + (c & 7), (c >> 3 & 15) - 10)) for c in range(256)]
    value[127] = value[255] = math.nan
    power = [math.ldexp(1.0, b - 127) for b in range(256)]
    return (torch.tensor(value, dtype=torch.float64, device=device),
            torch.tensor(power, dtype=torch.float64, device=device))
