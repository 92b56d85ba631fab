"""Token embedding and layer norm against plain implementations in 64 bits, on the GPU.

Tolerances count roundings: one of the result to its format (half a step: eps / 2 of the value, or half the least
subnormal), and of fp32 sums of n terms at most n * 2^-24 of the sum of their magnitudes."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mixed_precision_adam_amd as Z
    from mixed_precision_adam_amd.driver import LayerNorm, TokenEmbedding

DEV = "cuda:0"
U = 2.0**-24
FORMATS = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def matrix(rows, cols, dtype, gen, sigma=1.0, spare=0, shift=0):
    """Random rows with `spare` columns between them, `shift` elements into their buffer; what lies between is NaN."""
    buf = torch.full((rows * (cols + spare) + shift + 8,), float("nan"), dtype=dtype, device=DEV)
    out = buf[shift:shift + rows * (cols + spare)].view(rows, cols + spare)[:, :cols]
    out.copy_(torch.randn(rows, cols, generator=gen, device=DEV).mul_(sigma))
    return out, buf


def between(x, buf):
    """The bytes of x's buffer that are not x's."""
    keep = torch.ones(buf.numel(), dtype=torch.bool, device=DEV)
    at = (x.storage_offset() + torch.arange(x.shape[0], device=DEV)[:, None] * x.stride(0) +
          torch.arange(x.shape[1], device=DEV))
    keep[at.reshape(-1)] = False
    return buf[keep].view(torch.int16 if buf.element_size() == 2 else torch.int32).clone()


def half_step(value, dtype):
    f = torch.finfo(dtype)
    return value.abs() * (f.eps / 2) + f.tiny * f.eps / 2


def check(name, got, want, bound):
    off = (got.double() - want).abs()
    worst = (off - bound).max().item() if off.numel() else 0.0
    assert not off.isnan().any() and worst <= 0.0, f"{name}: {worst:.3g} over its bound, off {off.max().item():.3g}"


# ------------------------------------------------------------------ embedding


def texts(kind, tokens, vocab, rng):
    if kind == "same":
        return np.full(tokens, vocab // 2)
    if kind == "skewed":
        return np.minimum(np.exp(rng.random(tokens) * np.log(vocab + 1)).astype(np.int64) - 1, vocab - 1)
    if kind == "outside":
        return rng.integers(-vocab, 2 * vocab, tokens)
    return rng.integers(0, vocab, tokens)


@pytest.mark.parametrize("table_dt", FORMATS)
@pytest.mark.parametrize("out_dt", FORMATS)
@pytest.mark.parametrize("tokens,vocab,cols,spare,shift", [(1, 1, 1, 0, 0), (5, 70, 8, 0, 0), (300, 70, 31, 3, 1),
                                                            (2500, 513, 1600, 8, 0), (1030, 40, 2100, 0, 5)])
def test_embed_forward(table_dt, out_dt, tokens, vocab, cols, spare, shift):
    gen, rng = torch.Generator(DEV).manual_seed(tokens), np.random.default_rng(tokens)
    table, _ = matrix(vocab, cols, FORMATS[table_dt], gen, 0.02, spare, shift)
    out, buf = matrix(tokens, cols, FORMATS[out_dt], gen, 1.0, spare, shift)
    for kind, first, wide in (("any", 0, True), ("outside", vocab // 3, False)):
        ids = torch.from_numpy(texts(kind, tokens, vocab, rng)).to(DEV)
        ids = ids if wide else ids.int()
        rest = between(out, buf)
        TokenEmbedding(table, scale=1.7, first_row=first).forward(ids, out)
        at = ids.long() - first
        held = (at >= 0) & (at < vocab)
        want = table.double()[at.clamp(0, vocab - 1)] * np.float32(1.7) * held[:, None]
        check("out", out, want, half_step(want, out.dtype) + U * want.abs())
        assert torch.equal(between(out, buf), rest)


def embed_grad_reference(ids, first, out_grad, scale, old, vocab):
    """Sums and sums of magnitudes, in 64 bits, and how many tokens each row has."""
    at = ids.long() - first
    held = (at >= 0) & (at < vocab)
    g = out_grad.double()[held] * scale
    sums = torch.zeros(vocab, out_grad.shape[1], dtype=torch.float64, device=DEV).index_add_(0, at[held], g)
    size = torch.zeros_like(sums).index_add_(0, at[held], g.abs())
    many = torch.bincount(at[held], minlength=vocab)
    return (sums if old is None else sums + old.double()), size + (0 if old is None else old.double().abs()), many


@pytest.mark.parametrize("out_dt,grad_dt", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp16"), ("fp32", "fp32"),
                                            ("fp16", "fp16"), ("bf16", "fp32")])
@pytest.mark.parametrize("tokens,vocab,cols,spare,shift,kind", [
    (0, 5, 7, 0, 0, "any"), (1, 1, 1, 0, 0, "any"), (3, 200, 16, 0, 0, "outside"), (301, 130, 523, 1, 3, "skewed"),
    (512, 40, 64, 0, 0, "same"), (513, 40, 64, 0, 0, "same"), (513, 1, 9, 0, 1, "any"), (1000, 511, 40, 0, 0, "any"),
    (1700, 512, 24, 8, 0, "outside"), (4000, 50257, 72, 0, 0, "skewed"), (70_001, 300_000, 17, 0, 0, "any"),
    (40_000, 37, 1027, 2, 1, "skewed"), (9000, 3, 520, 0, 0, "any"), (280_000, 900, 8, 0, 0, "skewed"),
    (280_000, 2, 4, 0, 0, "same")])
def test_embed_grad(out_dt, grad_dt, tokens, vocab, cols, spare, shift, kind):
    gen, rng = torch.Generator(DEV).manual_seed(tokens + cols), np.random.default_rng(tokens)
    ids = torch.from_numpy(texts(kind, tokens, vocab, rng)).to(DEV)
    first = vocab // 4 if kind == "outside" else 0
    out_grad, _ = matrix(tokens, cols, FORMATS[out_dt], gen, 1e-2, spare, shift)
    if kind == "outside":  # what no row of the table asks for is not read
        at = ids - first
        out_grad[(at < 0) | (at >= vocab)] = float("nan")
    op = TokenEmbedding(torch.empty(vocab, cols, device=DEV), max_tokens=max(tokens, 1), scale=2.5, first_row=first)
    for accumulate in (False, True):
        grad, buf = matrix(vocab, cols, FORMATS[grad_dt], gen, 1e-2, spare, shift)
        old = grad.clone()
        rest = between(grad, buf)
        op.ws.fill_(0xA5)  # nothing is taken from an earlier call
        op.grad(ids if accumulate else ids.int(), out_grad, grad, accumulate=accumulate)
        want, size, many = embed_grad_reference(ids, first, out_grad, 2.5, old if accumulate else None, vocab)
        check("table_grad", grad, want, half_step(want, grad.dtype) + (many[:, None] + 2) * U * size)
        assert torch.equal(between(grad, buf), rest)
        bare = many == 0
        assert torch.equal(grad[bare], old[bare] if accumulate else torch.zeros_like(old[bare]))
        again = old.clone() if accumulate else torch.full_like(old, 3.0)
        op.grad(ids, out_grad, again, accumulate=accumulate)
        assert torch.equal(again, grad)  # one order for every sum


def test_embed_grad_of_fewer_tokens_than_the_workspace_is_for():
    """Past 2^18 tokens the chunks get longer and the workspace's edges fewer: a smaller call must fit all the same."""
    for most in (262_145, 300_000, 1 << 19):
        for n in (262_144, 262_145, 1000, 512):
            assert Z.zero_embed_grad_workspace_bytes(n, 100, 600) <= Z.zero_embed_grad_workspace_bytes(most, 100, 600)
    gen = torch.Generator(DEV).manual_seed(4)
    ids = torch.randint(0, 100, (262_144,), generator=gen, device=DEV)
    out_grad = torch.randn(262_144, 24, generator=gen, device=DEV)
    op = TokenEmbedding(torch.empty(100, 24, device=DEV), max_tokens=262_145)
    grad = torch.empty(100, 24, device=DEV)
    op.grad(ids, out_grad, grad)
    want, size, many = embed_grad_reference(ids, 0, out_grad, 1.0, None, 100)
    check("table_grad", grad, want, half_step(want, grad.dtype) + (many[:, None] + 2) * U * size)


# ------------------------------------------------------------------ layer norm

# A lane adds up to 64 terms, then 8 levels of lanes and wavefronts; the quotients and the root add a few.
GAMMA = 128 * U
ROWS = [(1, 1), (3, 8), (7, 511), (5, 512), (9, 777), (4, 1024), (33, 1600), (2, 2049), (3, 4104), (130, 5120),
        (3, 8192), (2, 8197), (1, 16384), (2500, 64)]


def norm_inputs(rows, cols, dtype, wide_weight, mean, spare, shift, seed=0):
    gen = torch.Generator(DEV).manual_seed(rows * 100_003 + cols + seed)
    x, _ = matrix(rows, cols, dtype, gen, 1.5, spare, shift)
    x.add_(0.5)
    wdt = torch.float32 if wide_weight else dtype
    weight = torch.randn(cols, generator=gen, device=DEV).mul_(0.2).add_(1.0).to(wdt)
    bias = torch.randn(cols, generator=gen, device=DEV).to(wdt) if mean else None
    return gen, x, weight, bias


@pytest.mark.parametrize("mean", [True, False])
@pytest.mark.parametrize("dt,wide_weight", [("bf16", False), ("bf16", True), ("fp16", False), ("fp32", False)])
@pytest.mark.parametrize("rows,cols", ROWS)
def test_layernorm_forward(rows, cols, dt, wide_weight, mean):
    spare, shift = (0, 0) if cols % 8 == 0 and rows % 2 else (3, 1)
    _, x, weight, bias = norm_inputs(rows, cols, FORMATS[dt], wide_weight, mean, spare, shift)
    out, buf = matrix(rows, cols, FORMATS[dt], torch.Generator(DEV), 1.0, spare, shift)
    rest = between(out, buf)
    mu, rstd = torch.full((rows,), 7.0, device=DEV), torch.zeros(rows, device=DEV)
    op = LayerNorm(weight, bias, eps=1e-3, mean=mean)
    op.forward(x, out, mu if mean else None, rstd)
    xd, w = x.double(), weight.double()
    m = xd.mean(1, keepdim=True) if mean else torch.zeros(rows, 1, dtype=torch.float64, device=DEV)
    r = ((xd - m).square().mean(1, keepdim=True) + 1e-3).rsqrt()
    h = (xd - m) * r
    level = xd.abs().mean(1, keepdim=True)
    want = h * w + (bias.double() if mean else 0.0)
    slack = GAMMA * ((h.abs() + r * level) * w.abs() + (bias.double().abs() if mean else 0.0))
    check("out", out, want, half_step(want, out.dtype) + slack)
    check("rstd", rstd, r[:, 0], GAMMA * r[:, 0] * (1 + (r * level)[:, 0] ** 2))
    if mean:
        check("mean", mu, m[:, 0], GAMMA * level[:, 0])
    assert torch.equal(between(out, buf), rest)
    bare = torch.empty_like(out)
    op.forward(x, bare)  # without the statistics
    assert torch.equal(bare, out)


def test_layernorm_of_a_far_mean():
    """The variance comes from the differences to the mean, so a mean of 1000 times the spread costs no more than its
    own rounding: 2^-24 * 1000 of the spread."""
    x = torch.randn(64, 1601, generator=torch.Generator(DEV).manual_seed(1), device=DEV) + 1000.0
    out, mu, rstd = torch.empty_like(x), torch.empty(64, device=DEV), torch.empty(64, device=DEV)
    LayerNorm(torch.ones(1601, device=DEV), eps=0.0).forward(x, out, mu, rstd)
    want = (x.double() - x.double().mean(1, keepdim=True)) / x.double().std(1, keepdim=True, unbiased=False)
    check("out", out, want, torch.full_like(want, 2 * GAMMA * 1000))


@pytest.mark.parametrize("mean", [True, False])
@pytest.mark.parametrize("dt,wide_weight,grad_dt", [("bf16", False, "bf16"), ("bf16", True, "fp32"),
                                                    ("fp16", False, "fp32"), ("fp32", False, "fp32"),
                                                    ("fp16", True, "fp16")])
@pytest.mark.parametrize("rows,cols", ROWS + [(0, 40), (5000, 264)])
def test_layernorm_grad(rows, cols, dt, wide_weight, grad_dt, mean):
    spare, shift = (0, 0) if cols % 8 == 0 and rows % 2 else (5, 3)
    gen, x, weight, bias = norm_inputs(rows, cols, FORMATS[dt], wide_weight, mean, spare, shift, 1)
    dy, _ = matrix(rows, cols, FORMATS[dt], gen, 0.1, spare, shift)
    xd, w, g = x.double(), weight.double(), dy.double()
    m = xd.mean(1, keepdim=True) if mean else torch.zeros(rows, 1, dtype=torch.float64, device=DEV)
    r = ((xd - m).square().mean(1, keepdim=True) + 1e-5).rsqrt()
    mu, rstd = m[:, 0].float(), r[:, 0].float()
    m, r = mu.double()[:, None], rstd.double()[:, None]
    h, d = (xd - m) * r, g * w
    along, level = (d * h).mean(1, keepdim=True), d.mean(1, keepdim=True) if mean else 0.0
    want = r * (d - level - h * along)
    slack = GAMMA * r * (d.abs() + d.abs().mean(1, keepdim=True) + h.abs() * (d * h).abs().mean(1, keepdim=True))
    op = LayerNorm(weight, bias, mean=mean)
    for accumulate in (False, True):
        dx, buf = matrix(rows, cols, FORMATS[dt], gen, 1.0, spare, shift)
        rest = between(dx, buf)
        dw, db = (torch.randn(cols, generator=gen, device=DEV).to(FORMATS[grad_dt]) for _ in range(2))
        old = dw.double(), db.double()
        if not mean:
            db = None
        op.ws.fill_(0xA5)
        op.grad(x, dy, mu if mean else None, rstd, dx, dw, db, accumulate=accumulate)
        if rows:
            check("x_grad", dx, want, half_step(want, dx.dtype) + slack)
        assert torch.equal(between(dx, buf), rest)
        for name, got, terms, before in (("weight_grad", dw, g * h, old[0]), ("bias_grad", db, g, old[1])):
            if got is None:
                continue
            total, size = terms.sum(0), terms.abs().sum(0)
            if accumulate:
                total, size = total + before, size + before.abs()
            check(name, got, total, half_step(total, got.dtype) + (rows + 4) * U * size)
    only = torch.empty_like(dw)
    op.grad(x, dy, mu, rstd, weight_grad=only)  # one of the three alone
    again = torch.empty_like(dx)
    op.grad(x, dy, mu, rstd, x_grad=again)
    assert torch.equal(again, dx)
    total = (g * h).sum(0)
    check("weight_grad", only, total, half_step(total, only.dtype) + (rows + 4) * U * (g * h).abs().sum(0))


def test_layernorm_grad_against_differences():
    """Central differences of the plain forward in 64 bits: their error is of the order step^2 = 1e-8, and far larger
    than 1e-4 of the gradients for any slip in a term."""
    gen = torch.Generator(DEV).manual_seed(3)
    rows, cols, step = 3, 24, 1e-4
    x, dy = (torch.randn(rows, cols, generator=gen, device=DEV) for _ in range(2))
    weight, bias = (torch.randn(cols, generator=gen, device=DEV) for _ in range(2))

    def loss(x, weight, bias, mean):
        m = x.mean(1, keepdim=True) if mean else 0.0
        h = (x - m) * ((x - m).square().mean(1, keepdim=True) + 1e-5).rsqrt()
        return ((h * weight + bias) * dy.double()).sum().item()

    for mean in (True, False):
        op = LayerNorm(weight, bias, mean=mean)
        out, mu, rstd = torch.empty_like(x), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
        op.forward(x, out, mu, rstd)
        grads = [torch.empty_like(x), torch.empty_like(weight), torch.empty_like(bias)]
        op.grad(x, dy, mu, rstd, *grads)
        point = [x.double(), weight.double(), bias.double()]
        for k, grad in enumerate(grads):
            for i in range(0, grad.numel(), 7):
                found = []
                for sign in (1, -1):
                    moved = [p.clone() for p in point]
                    moved[k].view(-1)[i] += sign * step
                    found.append(loss(*moved, mean))
                want = (found[0] - found[1]) / (2 * step)
                assert abs(grad.view(-1)[i].item() - want) <= 1e-4 * (1 + abs(want)), (mean, k, i)


@pytest.mark.parametrize("mean", [True, False])
def test_layernorm_without_gradients(mean):
    """The forward pass alone needs no workspace, and gives the same bits."""
    _, x, weight, bias = norm_inputs(33, 1600, torch.bfloat16, False, mean, 0, 0)
    outs = []
    for gradients in (True, False):
        out, mu, rstd = torch.empty_like(x), torch.zeros(33, device=DEV), torch.zeros(33, device=DEV)
        op = LayerNorm(weight, bias, mean=mean, gradients=gradients)
        assert (op.ws is None) == (not gradients)
        op.forward(x, out, mu, rstd)
        outs.append((out, mu, rstd))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    with pytest.raises(ValueError, match="without gradients"):
        op.grad(x, x, mu, rstd, torch.empty_like(x))


@pytest.mark.parametrize("mean", [True, False])
@pytest.mark.parametrize("rows,cols", [(33, 1600), (5, 777), (3, 8197), (2500, 64), (130, 5120)])
def test_layernorm_in_place(rows, cols, mean):
    """y over x, and x_grad over x or over y_grad: the bits of a call with memory of its own for each."""
    gen, x, weight, bias = norm_inputs(rows, cols, torch.bfloat16, False, mean, 3, 1)
    dy, _ = matrix(rows, cols, torch.bfloat16, gen, 0.1, 5, 2)
    op = LayerNorm(weight, bias, mean=mean)
    out, dx = torch.empty(rows, cols, dtype=x.dtype, device=DEV), torch.empty(rows, cols, dtype=x.dtype, device=DEV)
    mu, rstd = torch.zeros(rows, device=DEV), torch.zeros(rows, device=DEV)
    dw, dw2 = torch.zeros(cols, device=DEV), torch.zeros(cols, device=DEV)
    op.forward(x, out, mu, rstd)
    op.grad(x, dy, mu, rstd, dx, dw)
    for over in (0, 1):
        held = [t.clone() for t in (x, dy)]
        op.grad(*held, mu, rstd, held[over], dw2)
        assert torch.equal(held[over], dx) and torch.equal(dw2, dw)
    op.forward(x, x)
    assert torch.equal(x, out)
