"""Timed cases of the operators over lists of tensors, and their plain forms.

The operators work on many tensors at once, where they lie: the square-norm of a list of gradients
(``norm``), the AdamW update with fp32 states (``adamw``) and with moments held in 8 bits (``adamw8``),
and the conversion of the moments between fp32 and 8 bits (``pack``, ``unpack``).

A case names a list of tensors, the formats and the state's layout.  Tensors start at tile boundaries of flat
buffers (gradients, parameters, states), as gradient buckets and flat parameter buffers hold them, so the plain
forms work on whole buffers; a ``shift`` moves gradients and parameters off the 16-byte lines.  Padding between
tensors is zero and stays zero.

With ``own`` false, ``run`` computes in elementary torch operations; with ``own`` true it calls this
repository's package.  ``exact`` computes the same outputs in 64 bits.
"""
import math
import random

import torch

own = False

TILE = 1024    # elements per tile of the fp32 state: [master | m | v]
TILE8 = 4096   # elements per tile of the 8-bit state: [master | m codes | v codes | m scales | v scales]
BLOCK8 = 256   # elements that share one m scale and one v scale
TILE8_BYTES = 6 * TILE8 + 8 * (TILE8 // BLOCK8)
FLOATS = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
BETA1, BETA2, EPS = 0.9, 0.999, 1e-8
GROUPS = ((1e-4, 0.1), (2e-4, 0.0))  # (learning rate, weight decay): matrices, then vectors
LOSS_SCALE = 65536.0                 # fp16 gradients are stored multiplied by it
ROUNDING_SEED = 20240229
GOLDEN, MIX1, MIX2 = 0x9E3779B97F4A7C15, 0xBF58476D1CE4E5B9, 0x94D049BB133111EB  # SplitMix64
WEYL = 0x9E3779B9


def case(name, op, model, grad="bf16", param="bf16", layout="tiled", shift=0, step=100, world=1, rank=0, tensors=0,
         total=0):
    return {"name": name, "op": op, "model": model, "world": world, "rank": rank, "tensors": tensors, "total": total,
            "grad": grad, "param": param, "layout": layout, "shift": shift, "step": step}


def listed():
    gpt = dict(model="gpt2-1.5b", world=8)           # rank 0 of 8: 195M parameters in 47 pieces
    llama = dict(model="llama-7b", world=8, rank=3)  # rank 3 of 8: 842M parameters in 38 pieces
    return [
        # adapters or a tiny model: the launches are what it costs
        case("norm-small", "norm", "mixed", tensors=16, total=40_003),
        # a rank's pieces before clipping
        case("norm-gpt2", "norm", **gpt),
        # fp32 gradients, hundreds of ragged tensors off the 16-byte lines
        case("norm-ragged-fp32", "norm", "mixed", grad="fp32", shift=3, tensors=500, total=60_000_007),
        case("adamw-small", "adamw", "mixed", tensors=16, total=40_003, step=3),
        case("adamw-gpt2", "adamw", **gpt),
        # the optimizer's tensors as a training program keeps them: separate fp32 arrays, fp16 with a loss scale
        case("adamw-ragged-arrays", "adamw", "mixed", grad="fp16", param="fp16", layout="arrays", shift=3,
             tensors=500, total=60_000_007, step=1),
        case("adamw-llama", "adamw", grad="fp16", step=2000, **llama),
        # the 8-bit cases read the moments back after the step
        case("adamw8-small", "adamw8", "mixed", tensors=16, total=40_003, step=3),
        case("adamw8-ragged", "adamw8", "mixed", grad="fp32", param="fp32", shift=1, tensors=500, total=60_000_007),
        case("adamw8-llama", "adamw8", grad="fp16", step=2000, **llama),
        # moments into 8 bits (and what they then stand for); a checkpoint's read-back
        case("pack-gpt2", "pack", **gpt),
        case("unpack-ragged", "unpack", "mixed", layout="arrays", tensors=500, total=60_000_007),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    c = case("", rng.choice(("norm", "adamw", "adamw", "adamw8", "adamw8", "pack", "unpack")), "mixed",
             grad=rng.choice(("bf16", "fp16", "fp32")), param=rng.choice(("bf16", "fp16", "fp32")),
             layout=rng.choice(("tiled", "arrays")), shift=rng.randrange(8), step=spread(1, 5000),
             tensors=spread(1, 600), total=spread(3_000, 150_000_000) | 1)
    del c["name"]
    return c


# ------------------------------------------------------------------ the lists


def shard_pieces(numels, world, rank):
    """Pieces of tensors laid end to end that fall in one rank's equal share."""
    share = -(-sum(numels) // world)
    lo, hi, at, out = rank * share, (rank + 1) * share, 0, []
    for n in numels:
        a, b = max(at, lo), min(at + n, hi)
        if b > a:
            out.append(b - a)
        at += n
    return out


def sizes(c):
    """Elements of each tensor of the case's list."""
    if c["model"] == "gpt2-1.5b":
        d, block = 1600, [1600, 1600, 3 * 1600 * 1600, 4800, 1600 * 1600, 1600, 1600, 1600, 1600 * 6400, 6400,
                          6400 * 1600, 1600]
        return shard_pieces([50257 * d, 1024 * d] + block * 48 + [d, d], c["world"], c["rank"])
    if c["model"] == "llama-7b":
        d, f = 4096, 11008
        return shard_pieces([32000 * d] + ([d] + [d * d] * 4 + [d] + [d * f] * 3) * 32 + [d, 32000 * d], c["world"],
                            c["rank"])
    # a few large tensors, many small ones, any size from one element on
    rng = random.Random(1000 * c["tensors"] + c["total"])
    w = [math.exp(rng.uniform(0.0, math.log(1e4))) for _ in range(c["tensors"])]
    return [max(1, int(c["total"] * x / sum(w))) for x in w]


def tile_of(c):
    return TILE8 if c["op"] in ("adamw8", "pack", "unpack") else TILE


def plan(c):
    """(elements, offset in the flat buffers, group) of each tensor, and the flat buffers' size."""
    t, at, out = tile_of(c), 0, []
    for n in sizes(c):
        out.append((n, at, 0 if n > 8192 else 1))
        at += -(-n // t) * t
    return out, at


def hyper(c, group):
    """The group's update scalars, computed in 64 bits."""
    lr, wd = GROUPS[group]
    t = c["step"]
    return {"decay": 1 - lr * wd, "step_size": lr / (1 - BETA1**t), "bc2_sqrt": math.sqrt(1 - BETA2**t)}


def grad_scale(c):
    return 0.7 / (LOSS_SCALE if c["grad"] == "fp16" else 1.0)  # a clipped step


# ------------------------------------------------------------------ inputs


def prepare(c, seed):
    dev = "cuda"
    gen = torch.Generator(dev).manual_seed(seed)
    tensors, n = plan(c)
    s = {"case": c, "n": n}

    def normal():
        return torch.randn(n, generator=gen, device=dev)

    def clear(x, quiet=True):
        """Zeroes the padding and (embedding rows that no token met) every 64th block of 256."""
        if quiet:
            x.view(-1, 256)[5::64] = 0
        ends = [a for k, (m, o, _) in enumerate(tensors) for a in (o + m, tensors[k + 1][1] if k + 1 < len(tensors)
                                                                   else n)]
        for lo, hi in zip(ends[::2], ends[1::2]):
            if hi > lo:
                x[lo:hi] = 0
        return x

    def shifted(x, dtype):
        """The same values starting c["shift"] elements into a buffer of their own."""
        buf = torch.zeros(n + 8, dtype=dtype, device=dev)
        out = buf[c["shift"]:c["shift"] + n]
        out.copy_(x)
        return out

    if c["op"] in ("norm", "adamw", "adamw8"):
        g = normal().mul_(1e-3 * (LOSS_SCALE if c["grad"] == "fp16" else 1.0))
        g[torch.randint(n, (n // 1000 + 1,), generator=gen, device=dev)] *= 20.0  # a thousandth are outliers
        s["grad"] = shifted(clear(g), FLOATS[c["grad"]])
        del g
    if c["op"] == "norm":
        s["sq"] = torch.zeros(1, dtype=torch.float64, device=dev)
        s["flag"] = torch.zeros(1, dtype=torch.int32, device=dev)
    else:
        master = clear(normal().mul_(0.02), quiet=False)
    if c["op"] in ("adamw", "adamw8"):
        s["param"] = shifted(master, FLOATS[c["param"]])
    if c["op"] in ("adamw", "pack"):
        m = clear(normal().mul_(3e-4))
        v = clear(normal().square_().mul_(0.3).add_(0.05).mul_(1e-6))
        if c["layout"] == "tiled":
            s["state"] = torch.stack([x.view(-1, TILE) for x in (master, m, v)], dim=1)  # [tiles, 3, TILE]
            s["p"], s["m"], s["v"] = (s["state"][:, k] for k in range(3))
        else:
            s["p"], s["m"], s["v"] = (x.view(-1, TILE) for x in (master, m, v))
    if c["op"] == "pack":
        s["state8"] = torch.zeros(n // TILE8, TILE8_BYTES, dtype=torch.uint8, device=dev)
    if c["op"] in ("adamw8", "unpack"):
        s["state8"] = torch.zeros(n // TILE8, TILE8_BYTES, dtype=torch.uint8, device=dev)
        p, mc, vc, ms, vs = fields8(s["state8"])
        p.copy_(master.view(-1, TILE8))
        codes = clear(normal().mul_(120.0)).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        mc.copy_(codes.view(-1, TILE8))
        vc.copy_(clear(torch.randint(150, 256, (n,), generator=gen, device=dev, dtype=torch.int32))
                 .view(-1, TILE8))
        blocks = torch.rand(2, n // TILE8, TILE8 // BLOCK8, generator=gen, device=dev).add_(0.5)
        ms.copy_(blocks[0] * (1e-3 / 448))
        vs.copy_(blocks[1] * (4e-6 / 1.875))
    if c["op"] in ("adamw8", "pack", "unpack"):
        s["out"] = [torch.zeros(n, device=dev) for _ in range(2 if c["op"] == "adamw8" else 3)]  # moments; master
    groups = torch.zeros(n // tile_of(c), dtype=torch.int64)
    for size, off, group in tensors:
        groups[off // tile_of(c):off // tile_of(c) - (-size // tile_of(c))] = group
    s["groups"] = groups.to(dev)
    if own:
        keep_lists(s, tensors)
    return s


def fields8(state8):
    """The parts of a [tiles, bytes] 8-bit state: master, m codes, v codes, m scales, v scales."""
    a, b = 4 * TILE8, TILE8 // BLOCK8
    return (state8[:, :a].view(torch.float32), state8[:, a:a + TILE8], state8[:, a + TILE8:a + 2 * TILE8],
            state8[:, a + 2 * TILE8:a + 2 * TILE8 + 4 * b].view(torch.float32),
            state8[:, a + 2 * TILE8 + 4 * b:].view(torch.float32))


def keep_lists(s, tensors):
    """What a training program keeps for its lists: the plans and the hyper-parameters of the groups."""
    import mixed_precision_adam_amd as Z
    from mixed_precision_adam_amd.driver import TensorList

    c = s["case"]
    numels = [n for n, _, _ in tensors]
    groups = [g for _, _, g in tensors]

    def cut(flat):
        return [flat[o:o + n] for n, o, _ in tensors]

    def fp32(flats):
        return {k: cut(f) for k, f in zip(("master", "m", "v"), flats) if f is not None}

    if c["op"] == "norm":
        s["list"] = TensorList(numels, cut(s["grad"]))
    if c["op"] in ("adamw", "pack"):
        if c["layout"] == "tiled":
            held = {"state": [s["state"][o // TILE:o // TILE - (-n // TILE)].view(-1) for n, o, _ in tensors]}
        else:
            held = fp32([x.view(-1) for x in (s["p"], s["m"], s["v"])])
        more = (cut(s["grad"]), cut(s["param"])) if c["op"] == "adamw" else ()
        s["list"] = TensorList(numels, *more, groups=groups, n_groups=len(GROUPS), **held)
    if "state8" in s:
        held = {"state8": [s["state8"][o // TILE8:o // TILE8 - (-n // TILE8)].view(-1) for n, o, _ in tensors]}
        more = (cut(s["grad"]), cut(s["param"])) if c["op"] == "adamw8" else ()
        s["list8"] = TensorList(numels, *more, groups=groups, n_groups=len(GROUPS), **held)
        s["out_list"] = TensorList(numels, **fp32([None] * (3 - len(s["out"])) + s["out"]))
    s["hparams"] = Z.zero_list_hparams([
        dict(lr=lr, beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=wd, grad_scale=grad_scale(c), step=c["step"])
        for lr, wd in GROUPS])


# ------------------------------------------------------------------ one pass


def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    op = s["case"]["op"]
    if op == "norm":
        s["list"].grad_sqnorm(s["sq"], s["flag"])
        return {"sqnorm": s["sq"], "nonfinite": s["flag"]}
    if op == "adamw":
        s["list"].adamw(s["hparams"])
        return {"master": s["p"], "m": s["m"], "v": s["v"], "param": s["param"]}
    if op == "adamw8":
        s["list8"].adamw(s["hparams"], seed=ROUNDING_SEED)
        s["list8"].unpack8(s["out_list"])
        return {"master": fields8(s["state8"])[0], "m": s["out"][0], "v": s["out"][1], "param": s["param"]}
    if op == "pack":
        s["list"].pack8(s["list8"])
    s["list8"].unpack8(s["out_list"])
    return dict(zip(("master", "m", "v"), s["out"]))


def run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "norm":
        x = s["grad"].double()
        s["sq"][0] = x.square().sum()
        s["flag"][0] = (~torch.isfinite(x)).any()
        return {"sqnorm": s["sq"], "nonfinite": s["flag"]}
    if op == "adamw":
        g = s["grad"].view(-1, TILE).float()
        p, m, v = update(c, s["groups"], g, s["p"], s["m"], s["v"])
        s["p"].copy_(p)
        s["m"].copy_(m)
        s["v"].copy_(v)
        s["param"].copy_(p.view(-1))
        return {"master": s["p"], "m": s["m"], "v": s["v"], "param": s["param"]}
    p8, mc, vc, ms, vs = fields8(s["state8"])
    if op == "pack":
        p8.copy_(s["p"].reshape(-1, TILE8))
        encode8(s["state8"], s["m"].reshape(-1, BLOCK8), s["v"].reshape(-1, BLOCK8), 0x80000, 0x80000)
    if op == "adamw8":
        m, v = decode8(s["state8"])
        g = s["grad"].view(-1, TILE8).float()
        p, m, v = update(c, s["groups"], g, p8, m.view(-1, TILE8), v.view(-1, TILE8))
        p8.copy_(p)
        s["param"].copy_(p.view(-1))
        r = dither(s["n"] // BLOCK8, c["step"], p.device)
        encode8(s["state8"], m.view(-1, BLOCK8), v.view(-1, BLOCK8), r >> 12, r & 0xFFFFF)
        del p, m, v, g, r
    m, v = decode8(s["state8"])
    if op == "adamw8":
        return {"master": p8, "m": m.view(-1), "v": v.view(-1), "param": s["param"]}
    return {"master": p8.reshape(-1), "m": m.view(-1), "v": v.view(-1)}


def update(c, groups, g, p, m, v):
    """AdamW, every operation rounded to fp32; rows are tiles, whose scalars are those of their tensor's group."""
    rows = [torch.tensor([hyper(c, k)[w] for k in range(len(GROUPS))], device=g.device)[groups][:, None]
            for w in ("decay", "step_size")]
    g = g * grad_scale(c)
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + (g * g) * (1 - BETA2)
    d = v.sqrt() / hyper(c, 0)["bc2_sqrt"] + EPS
    return p * rows[0] - (m / d) * rows[1], m, v


def e5m3_values(device):
    """What the codes of the second moment stand for: 3 bits of fraction, 5 of exponent, no sign, up to 1.875."""
    code = torch.arange(256, device=device)
    e, f = code >> 3, (code & 7).float()
    return torch.where(e > 0, (1 + f / 8) * torch.exp2(e.float() - 31), f / 8 * 2.0**-30)


def decode8(state8):
    """(m, v) in fp32, one row a block."""
    _, mc, vc, ms, vs = fields8(state8)
    m = mc.reshape(-1, BLOCK8).view(torch.float8_e4m3fn).float() * ms.reshape(-1, 1)
    v = e5m3_values(vc.device)[vc.reshape(-1, BLOCK8).int()] * vs.reshape(-1, 1)
    return m, v


def encode8(state8, m, v, dither_m, dither_v):
    """Moments (one row a block) into codes and scales: the largest of a block takes the largest code, the others are
    rounded down after the dither (in 2^-20 of a step) is added."""
    _, mc, vc, ms, vs = fields8(state8)
    for x, top, low, most, codes, scales, add in ((m, 448.0, 2.0**-120, 126, mc, ms, dither_m),
                                                  (v, 1.875, 2.0**-96, 255, vc, vs, dither_v)):
        peak = x.abs().amax(1, keepdim=True)
        some = ~(peak < 2.0**-110)  # a block below is held as zeros
        scale = torch.where(some, peak * (1 / top), 0.0)
        inverse = torch.where(some, torch.full_like(peak, top) / peak, 0.0)
        # scaled so that the code is the top bits of the fp32 pattern, subnormals included
        bits = ((x.abs() * inverse) * low).view(torch.int32)
        code = ((bits + add) >> 20).clamp_(max=most)
        if top == 448.0:
            code = code | ((x.view(torch.int32) >> 24) & 0x80)
        else:
            code = torch.maximum(code, ((x > 0) & some).to(code.dtype))  # a second moment that is not zero stays so
        codes.copy_(code.view(-1, TILE8))
        scales.copy_(scale.view(scales.shape))


def mix64(z):
    z = (z ^ ((z >> 30) & 0x3FFFFFFFF)) * signed(MIX1)
    z = (z ^ ((z >> 27) & 0x1FFFFFFFFF)) * signed(MIX2)
    return z ^ ((z >> 31) & 0x1FFFFFFFF)


def signed(x):
    x &= (1 << 64) - 1
    return x - (1 << 64) if x >> 63 else x


def dither(blocks, step, device):
    """32 bits for each element: a hash of the seed, the step and the block, then a Weyl sequence in the block."""
    base = mix64(torch.tensor(signed(ROUNDING_SEED + step * GOLDEN), device=device))
    key = mix64(base + (torch.arange(blocks, device=device) + 1) * signed(GOLDEN))
    return (key[:, None] + torch.arange(BLOCK8, device=device) * WEYL) & 0xFFFFFFFF


# ------------------------------------------------------------------ work and 64-bit results


def work(c):
    n = sum(sizes(c))
    moments8 = 2 * n + 8 * sum(-(-x // BLOCK8) for x in sizes(c))  # codes and scales
    if c["op"] == "norm":
        return {"bytes": n * BYTES[c["grad"]], "flops": 2 * n}
    if c["op"] == "adamw":
        return {"bytes": n * (24 + BYTES[c["grad"]] + BYTES[c["param"]]), "flops": 16 * n}
    if c["op"] == "adamw8":  # the step, then the moments read back as fp32
        step = n * (8 + BYTES[c["grad"]] + BYTES[c["param"]]) + 2 * moments8
        return {"bytes": step + moments8 + 8 * n, "flops": 40 * n}
    unpack = 4 * n + moments8 + 12 * n
    pack = 12 * n + 4 * n + moments8
    return {"bytes": unpack + (pack if c["op"] == "pack" else 0), "flops": (20 if c["op"] == "pack" else 2) * n}


def exact(c, seed):
    s = prepare(c, seed)
    tensors, _ = plan(c)
    if c["op"] == "norm":
        parts = [s["grad"][o:o + n].double() for n, o, _ in tensors]
        total = math.fsum(float(torch.dot(x, x)) for x in parts)
        bad = any(bool((x != x).any() or x.abs().max() == math.inf) for x in parts)
        return {"sqnorm": torch.tensor([total], dtype=torch.float64), "nonfinite": torch.tensor([int(bad)])}
    if c["op"] == "pack":
        # The master is carried over as it is.  A moment whose value lies within an fp32 rounding of the middle of
        # two codes takes either: 64 bits do not say which.
        return {"master": s["p"].reshape(-1).double(), "m": None, "v": None}
    if "state8" in s:
        p8, mc, vc, ms, vs = fields8(s["state8"])
        mag = (mc & 127).long()
        e, f = (mag >> 3).double(), (mag & 7).double()
        size = torch.where(mag < 8, torch.ldexp(f, torch.full_like(e, -9.0)), torch.ldexp(8 + f, e - 10))
        m0 = size * (1 - 2 * (mc >> 7).double()) * ms.double().repeat_interleave(BLOCK8, 1)
        e, f = (vc >> 3).double(), (vc & 7).double()
        size = torch.where(vc < 8, torch.ldexp(f, torch.full_like(e, -33.0)), torch.ldexp(8 + f, e - 34))
        v0 = size * vs.double().repeat_interleave(BLOCK8, 1)
        p0, m0, v0 = p8.double().reshape(-1), m0.reshape(-1), v0.reshape(-1)
        if c["op"] == "unpack":
            return {"master": p0, "m": m0, "v": v0}
    else:
        p0, m0, v0 = (x.reshape(-1).double() for x in (s["p"], s["m"], s["v"]))
    t = c["step"]
    for n, o, k in tensors:
        lr, wd = GROUPS[k]
        at = slice(o, o + n)
        g = s["grad"][at].double() * grad_scale(c)
        m0[at] = m0[at].lerp(g, 1 - BETA1)
        v0[at] = v0[at].lerp(g.square(), 1 - BETA2)
        step = (m0[at] / (1 - BETA1**t)) / ((v0[at] / (1 - BETA2**t)).sqrt() + EPS)
        p0[at] -= lr * (wd * p0[at] + step)
    if c["op"] == "adamw8":
        # The new moments are rounded stochastically at positions that fp32 reaches a few roundings away from where
        # 64 bits do: a value next to a step's border takes either code, and no 64-bit value says which.
        return {"master": p0, "m": None, "v": None, "param": p0.clone()}
    return {"master": p0, "m": m0, "v": v0, "param": p0.clone()}
