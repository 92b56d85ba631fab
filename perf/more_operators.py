"""Timed cases of the operators at a language model's two ends and its norms, and their plain forms.

They are where the gradients come from that the lists of tensors step: the token embedding (``embed``, and the table's
gradient ``embed_grad``), layer norm with and without the mean (``norm``, ``norm_grad``) and the softmax cross entropy
of the output head over the vocabulary (``loss``: losses alone, or with the gradients of the hidden rows and of the
table, times the loss scale).

With ``own`` false, ``run`` computes in elementary torch operations; with ``own`` true it calls this
repository's package.  ``exact`` computes the same outputs in 64 bits.
"""
import math

import torch

own = False

FLOATS = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
IGNORED = -100  # the label of a position that does not count
MOST_PRODUCT = 4096 * 32000 * 4096  # tokens x vocabulary x columns of the largest loss


def case(name, op, tokens, cols, vocab=0, dtype="bf16", grad="bf16", first=0, rows=0, wide_ids=True, scale=1.0,
         mean=True, accumulate=False, gradients=True, ignored=0.0, loss_scale=1.0, spare=0):
    """``rows`` of the vocabulary from ``first`` on are held (0: all); ``grad``: the format of a weight's gradient;
    ``spare``: unused columns between two rows of the large operands."""
    return {"name": name, "op": op, "tokens": tokens, "cols": cols, "vocab": vocab, "dtype": dtype, "grad": grad,
            "first": first, "rows": rows or vocab, "wide_ids": wide_ids, "scale": scale, "mean": mean,
            "accumulate": accumulate, "gradients": gradients, "ignored": ignored, "loss_scale": loss_scale,
            "spare": spare}


def listed():
    gpt2 = dict(cols=1600, vocab=50257)
    llama7b = dict(cols=4096, vocab=32000)
    llama13b = dict(cols=5120, vocab=32000)
    return [
        # one token for each of 8 sequences being written
        case("embed-tokens", "embed", 8, scale=40.0, **gpt2),
        # a micro-batch of 8 sequences of 2048 tokens
        case("embed-llama", "embed", 16384, wide_ids=False, **llama7b),
        # a short odd sequence, added to the gradient that the tied head left
        case("embed-grad-short", "embed_grad", 301, accumulate=True, scale=40.0, **gpt2),
        # 8 sequences of the whole context
        case("embed-grad-gpt2", "embed_grad", 8192, wide_ids=False, **gpt2),
        # a rank that holds the upper half of the vocabulary; fp32 gradient over micro-batches
        case("embed-grad-slice", "embed_grad", 32769, dtype="fp16", grad="fp32", first=16000, rows=16000,
             accumulate=True, **llama13b),
        case("norm-tokens", "norm", 8, 1600),
        case("norm-gpt2", "norm", 16384, 1600),
        case("norm-grad-gpt2", "norm_grad", 16384, 1600),
        # Llama's norm, fp16, fp32 gradient over micro-batches, an odd number of rows
        case("norm-grad-llama", "norm_grad", 8191, 5120, dtype="fp16", grad="fp32", mean=False, accumulate=True),
        # the score of a short text
        case("loss-score", "loss", 33, gradients=False, **gpt2),
        # 4 sequences of the whole context, half a batch's prompts left out
        case("loss-gpt2", "loss", 4096, ignored=0.25, **gpt2),
        case("loss-llama", "loss", 4096, dtype="fp16", grad="fp16", loss_scale=8192.0, ignored=0.01, **llama7b),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    op = rng.choice(("embed", "embed_grad", "embed_grad", "norm", "norm_grad", "loss", "loss"))
    dtype = rng.choice(("bf16", "fp16") if op == "loss" else ("bf16", "fp16", "fp32"))
    grad = dtype if op == "loss" else rng.choice((dtype, "fp32"))
    cols = spread(48, 5120)
    cols = rng.choice((cols, cols // 8 * 8, cols | 1))
    tokens = spread(1, 16384) if op == "loss" else spread(1, 32769)
    vocab, first, rows = 0, 0, 0
    if op not in ("norm", "norm_grad"):
        vocab = spread(500, 60_000)
        if op == "loss":
            tokens = min(tokens, MOST_PRODUCT // (vocab * cols))
        elif rng.random() < 0.3:
            rows = max(1, vocab // rng.choice((2, 4, 8)))
            first = rng.randrange(vocab - rows + 1)
    c = case("", op, tokens, cols, vocab, dtype, grad, first, rows, rng.random() < 0.5,
             rng.choice((1.0, math.sqrt(cols))), rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.7,
             rng.choice((0.0, 0.05, 0.5)), 1024.0 if dtype == "fp16" else 1.0, rng.choice((0, 0, 8, 3)))
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs


def prepare(c, seed):
    dev = "cuda"
    gen = torch.Generator(dev).manual_seed(seed)
    tokens, cols, dtype, grad = c["tokens"], c["cols"], FLOATS[c["dtype"]], FLOATS[c["grad"]]
    s = {"case": c}

    def rows(n, like=dtype, width=cols):
        return torch.zeros(n, width + c["spare"], dtype=like, device=dev)[:, :width]

    def normal(n, sigma, like=dtype):
        return rows(n, like).copy_(torch.randn(n, cols, generator=gen, device=dev).mul_(sigma))

    def words():
        """Tokens as texts hold them: the k-th most frequent about 1/k as often as the first."""
        u = torch.rand(tokens, generator=gen, device=dev, dtype=torch.float64)
        rank = torch.exp(u * math.log(c["vocab"] + 1)).long().sub_(1).clamp_(0, c["vocab"] - 1)
        step = next(p for p in (7919, 7907, 7901) if c["vocab"] % p)  # frequent words lie all over the table
        return (rank * step + 11) % c["vocab"]

    if c["op"] in ("embed", "embed_grad"):
        s["ids"] = words() if c["wide_ids"] else words().int()
    if c["op"] == "embed":
        s["table"], s["out"] = normal(c["rows"], 0.02), rows(tokens)
    if c["op"] == "embed_grad":
        s["out_grad"] = normal(tokens, 1e-3)
        s["table_grad"] = normal(c["rows"], 1e-3, grad) if c["accumulate"] else rows(c["rows"], grad)
    if c["op"] in ("norm", "norm_grad"):
        size = torch.rand(tokens, 1, generator=gen, device=dev).mul_(3.0).add_(0.3)
        s["x"] = rows(tokens).copy_(normal(tokens, 1.0, torch.float32).add_(0.1).mul_(size))
        s["weight"] = torch.randn(cols, generator=gen, device=dev).mul_(0.1).add_(1.0).to(dtype)
        s["bias"] = torch.randn(cols, generator=gen, device=dev).mul_(0.1).to(dtype) if c["mean"] else None
        s["out"] = rows(tokens)
        s["mean"] = torch.zeros(tokens, device=dev) if c["mean"] else None
        s["rstd"] = torch.zeros(tokens, device=dev)
    if c["op"] == "norm_grad":
        x = s["x"].double()
        mu = x.mean(1) if c["mean"] else torch.zeros(tokens, dtype=torch.float64, device=dev)
        s["rstd"].copy_((x - mu[:, None]).square().mean(1).add(1e-5).rsqrt())
        if c["mean"]:
            s["mean"].copy_(mu)
        del x
        s["out_grad"], s["x_grad"] = normal(tokens, 1e-2), rows(tokens)
        s["weight_grad"] = torch.randn(cols, generator=gen, device=dev).mul_(0.1).to(grad)
        s["bias_grad"] = torch.randn(cols, generator=gen, device=dev).mul_(0.1).to(grad) if c["mean"] else None
    if c["op"] == "loss":
        s["table"] = normal(c["vocab"], 0.02)
        s["labels"] = words()
        # hidden rows as a norm leaves them, from indifferent to sure of their word
        sure = torch.rand(tokens, 1, generator=gen, device=dev).mul_(18.0 / (0.02**2 * cols))
        x = s["table"][s["labels"]].float().mul_(sure) + normal(tokens, 1.0, torch.float32)
        s["x"] = rows(tokens).copy_(x)
        del x
        s["labels"][torch.rand(tokens, generator=gen, device=dev) < c["ignored"]] = IGNORED
        if not c["wide_ids"]:
            s["labels"] = s["labels"].int()
        s["losses"] = torch.zeros(tokens, device=dev)
        s["loss"] = torch.zeros(1, device=dev)
        s["count"] = torch.zeros(1, dtype=torch.int64, device=dev)
        if c["gradients"]:
            s["x_grad"] = rows(tokens)
            s["table_grad"] = normal(c["vocab"], 1e-3) if c["accumulate"] else rows(c["vocab"])
        s["step_state"] = torch.zeros(16, dtype=torch.float64, device=dev)  # its first value is the loss scale
        s["step_state"][0] = c["loss_scale"]
    if own:
        keep(s)
    return s


def keep(s):
    """What a training program keeps between its steps: the operators, with their workspaces."""
    from mixed_precision_adam_amd.driver import LayerNorm, LossHead, TokenEmbedding

    c = s["case"]
    if c["op"] == "embed":
        s["embedding"] = TokenEmbedding(s["table"], scale=c["scale"], first_row=c["first"])
    if c["op"] == "embed_grad":  # the parameter itself is not read
        table = torch.empty(c["rows"], c["cols"], dtype=FLOATS[c["dtype"]], device=s["ids"].device)
        s["embedding"] = TokenEmbedding(table, max_tokens=c["tokens"], scale=c["scale"], first_row=c["first"])
    if c["op"] in ("norm", "norm_grad"):
        s["norm"] = LayerNorm(s["weight"], s["bias"], eps=1e-5, mean=c["mean"])
    if c["op"] == "loss":
        s["head"] = LossHead(s["table"], max_tokens=c["tokens"], gradients=c["gradients"])


# ------------------------------------------------------------------ one pass


def run(s):
    return run_own(s) if own else run_plain(s)


def outputs(s):
    names = {"embed": ("out",), "embed_grad": ("table_grad",), "norm": ("out", "mean", "rstd"),
             "norm_grad": ("x_grad", "weight_grad", "bias_grad"),
             "loss": ("losses", "loss", "count", "x_grad", "table_grad")}[s["case"]["op"]]
    return {k: s[k] for k in names if s.get(k) is not None}


def run_own(s):
    c = s["case"]
    if c["op"] == "embed":
        s["embedding"].forward(s["ids"], s["out"])
    elif c["op"] == "embed_grad":
        s["embedding"].grad(s["ids"], s["out_grad"], s["table_grad"], accumulate=c["accumulate"])
    elif c["op"] == "norm":
        s["norm"].forward(s["x"], s["out"], s["mean"], s["rstd"])
    elif c["op"] == "norm_grad":
        s["norm"].grad(s["x"], s["out_grad"], s["mean"], s["rstd"], s["x_grad"], s["weight_grad"], s["bias_grad"],
                       accumulate=c["accumulate"])
    elif c["gradients"]:
        s["head"].grad(s["x"], s["labels"], s["losses"], s["loss"], s["count"], s["x_grad"], s["table_grad"],
                       accumulate=c["accumulate"], step_state=s["step_state"])
    else:
        s["head"].forward(s["x"], s["labels"], s["losses"], s["loss"], s["count"])
    return outputs(s)


def run_plain(s):
    c = s["case"]
    if c["op"] == "embed":
        at, held = place(c, s["ids"])
        s["out"].copy_(s["table"][at].float() * (held * c["scale"])[:, None])
    elif c["op"] == "embed_grad":
        at, held = place(c, s["ids"])
        total = torch.zeros(c["rows"], c["cols"], device=at.device)
        total.index_add_(0, at, s["out_grad"].float() * (held * c["scale"])[:, None])
        s["table_grad"].copy_(s["table_grad"] + total if c["accumulate"] else total)
    elif c["op"] == "norm":
        x = s["x"].float()
        if c["mean"]:
            s["mean"].copy_(x.mean(1))
            x = x - s["mean"][:, None]
        s["rstd"].copy_((x.square().mean(1) + 1e-5).rsqrt())
        y = x * s["rstd"][:, None] * s["weight"].float()
        s["out"].copy_(y + s["bias"].float() if c["mean"] else y)
    elif c["op"] == "norm_grad":
        x, dy, r = s["x"].float(), s["out_grad"].float(), s["rstd"][:, None]
        xhat = (x - s["mean"][:, None]) * r if c["mean"] else x * r
        d = dy * s["weight"].float()
        dx = d - xhat * (d * xhat).mean(1, keepdim=True)
        if c["mean"]:
            dx = dx - d.mean(1, keepdim=True)
        s["x_grad"].copy_(dx * r)
        for name, total in (("weight_grad", (dy * xhat).sum(0)), ("bias_grad", dy.sum(0))):
            if s[name] is not None:
                s[name].copy_(s[name] + total if c["accumulate"] else total)
    else:
        plain_loss(s)
    return outputs(s)


def place(c, ids):
    """The row of the held slice for each token (any one for the others), and whether it is held."""
    at = ids.long() - c["first"]
    held = ((at >= 0) & (at < c["rows"])).float()
    return at.clamp(0, c["rows"] - 1), held


def plain_loss(s):
    c = s["case"]
    x, w = s["x"].float(), s["table"].float()
    z = x @ w.t()
    counted = (s["labels"] >= 0) & (s["labels"] < c["vocab"])
    label = s["labels"].long().clamp(0, c["vocab"] - 1)[:, None]
    top = z.amax(1, keepdim=True)
    p = (z - top).exp()
    total = p.sum(1, keepdim=True)
    s["losses"].copy_(torch.where(counted, (total.log() + top - z.gather(1, label))[:, 0], 0.0))
    s["count"].copy_(counted.sum())
    many = s["count"].clamp(min=1).float()
    s["loss"].copy_(s["losses"].sum() / many)
    if not c["gradients"]:
        return
    p /= total
    p.scatter_add_(1, label, torch.full_like(total, -1.0))
    p *= (counted / many * s["step_state"][:1].float())[:, None]
    s["x_grad"].copy_(p @ w)
    total = p.t() @ x
    s["table_grad"].copy_(s["table_grad"] + total if c["accumulate"] else total)


# ------------------------------------------------------------------ work and 64-bit results


def work(c):
    t, d, e, g = c["tokens"], c["cols"], BYTES[c["dtype"]], BYTES[c["grad"]]
    ids = t * (8 if c["wide_ids"] else 4)
    held = t * c["rows"] // max(1, c["vocab"])  # tokens whose row is held
    if c["op"] == "embed":
        return {"bytes": ids + (min(held, c["rows"]) + t) * d * e, "flops": held * d}
    if c["op"] == "embed_grad":  # added: the rows that tokens meet (about half as many as tokens); else every row
        met = 2 * min(held // 2 + 1, c["rows"]) if c["accumulate"] else c["rows"]
        return {"bytes": ids + held * d * e + met * d * g, "flops": 2 * held * d}
    if c["op"] == "norm":
        return {"bytes": 2 * t * d * e + 2 * d * e + 8 * t, "flops": 8 * t * d}
    if c["op"] == "norm_grad":
        return {"bytes": 3 * t * d * e + 2 * d * (e + g) + 8 * t, "flops": 14 * t * d}
    one = (t + c["vocab"]) * d
    parts = 2 + int(c["accumulate"]) * c["vocab"] * d / one if c["gradients"] else 1
    return {"bytes": parts * one * e + 12 * t, "flops": (6 if c["gradients"] else 2) * t * c["vocab"] * d}


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "embed":
        out = torch.zeros(c["tokens"], c["cols"], dtype=torch.float64, device=s["ids"].device)
        ids = s["ids"].long()
        held = (ids >= c["first"]) & (ids < c["first"] + c["rows"])
        out[held] = s["table"][ids[held] - c["first"]].double() * c["scale"]
        return {"out": out}
    if c["op"] == "embed_grad":
        ids, order = s["ids"].long().sort(stable=True)
        runs, sizes = ids.unique_consecutive(return_counts=True)
        ends = sizes.cumsum(0)
        sums = torch.cat([torch.zeros(1, c["cols"], dtype=torch.float64, device=ids.device),
                          s["out_grad"].double()[order].cumsum(0)])
        sums = (sums[ends] - sums[ends - sizes]) * c["scale"]
        held = (runs >= c["first"]) & (runs < c["first"] + c["rows"])
        grad = s["table_grad"].double() if c["accumulate"] else torch.zeros(
            c["rows"], c["cols"], dtype=torch.float64, device=ids.device)
        grad[runs[held] - c["first"]] += sums[held]
        return {"table_grad": grad}
    if c["op"] == "norm":
        x = s["x"].double()
        mu = x.sum(1) / c["cols"] if c["mean"] else x.new_zeros(c["tokens"])
        rstd = ((x - mu[:, None]) ** 2).sum(1).div(c["cols"]).add(1e-5) ** -0.5
        y = (x - mu[:, None]) * rstd[:, None] * s["weight"].double()
        if not c["mean"]:
            return {"out": y, "rstd": rstd}
        return {"out": y + s["bias"].double(), "mean": mu, "rstd": rstd}
    if c["op"] == "norm_grad":
        x, dy, w, r = s["x"].double(), s["out_grad"].double(), s["weight"].double(), s["rstd"].double()[:, None]
        xhat = (x - s["mean"].double()[:, None]) * r if c["mean"] else x * r
        along = (dy * w * xhat).sum(1, keepdim=True) / c["cols"]
        level = (dy @ w)[:, None] / c["cols"] if c["mean"] else 0.0
        found = {"x_grad": (dy * w - level - xhat * along) * r, "weight_grad": (dy.t() * xhat.t()).sum(1)}
        if c["mean"]:
            found["bias_grad"] = torch.ones_like(x[:, 0]) @ dy
        if c["accumulate"]:
            found = {k: v if k == "x_grad" else v + s[k].double() for k, v in found.items()}
        return found
    x, w, labels = s["x"].double(), s["table"].double(), s["labels"].long()
    rows = torch.nonzero((labels >= 0) & (labels < c["vocab"]))[:, 0]  # those that count
    losses, dx, dw = torch.zeros_like(x[:, 0]), torch.zeros_like(x), torch.zeros_like(w)
    factor = c["loss_scale"] / max(1, len(rows))
    for some in rows.split(1024):
        z = x[some] @ w.T
        k = torch.arange(len(some), device=z.device)
        lse = torch.logsumexp(z, 1)
        losses[some] = lse - z[k, labels[some]]
        if c["gradients"]:
            g = torch.exp(z - lse[:, None])
            g[k, labels[some]] = torch.expm1(-losses[some])
            dx[some] = (g @ w) * factor
            dw += (g.T @ x[some]) * factor
    found = {"losses": losses, "loss": losses.sum().view(1) / max(1, len(rows)),
             "count": torch.tensor([len(rows)], device=x.device)}
    if c["gradients"]:
        found |= {"x_grad": dx, "table_grad": dw + s["table_grad"].double() if c["accumulate"] else dw}
    return found
