"""The operators at a model's ends with the steps that take their gradients, as a training program runs them: a language
model of one tied table and one layer norm, trained by a ListDecision, on the GPU."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mixed_precision_adam_amd as Z
    from mixed_precision_adam_amd.driver import (AdamWConfig, LayerNorm, ListDecision, LossHead, TensorList,
                                                 TokenEmbedding)

DEV = "cuda:0"


class Model:
    """The model, its gradients and its optimizer state.  Everything that a step touches has one place in memory."""

    def __init__(self, dtype, vocab, cols, tokens, loss_scale=1.0, growth_interval=1000, seed=0):
        gen = torch.Generator(DEV).manual_seed(seed)
        self.vocab, self.cols, self.tokens = vocab, cols, tokens
        self.scale = math.sqrt(cols)

        def normal(*shape):
            return torch.randn(*shape, generator=gen, device=DEV)

        self.params = [(normal(vocab, cols) * 0.05).to(dtype), (1 + 0.1 * normal(cols)).to(dtype),
                       (0.1 * normal(cols)).to(dtype)]
        self.grads = [torch.zeros_like(p) for p in self.params]
        self.state = {"master": [p.float().view(-1) for p in self.params]}
        for k in ("m", "v"):
            self.state[k] = [torch.zeros_like(p) for p in self.state["master"]]
        self.list = TensorList([p.numel() for p in self.params], [g.view(-1) for g in self.grads],
                               [p.view(-1) for p in self.params], **self.state)
        self.config = AdamWConfig(lr=1e-2, max_norm=1.0)
        self.decision = ListDecision(self.list, [self.config], loss_scale=loss_scale, growth_interval=growth_interval)
        table, weight, bias = self.params
        self.embedding = TokenEmbedding(table, max_tokens=tokens, scale=self.scale)
        self.norm = LayerNorm(weight, bias)
        self.head = LossHead(table, max_tokens=tokens)
        self.x, self.h, self.dh, self.dx = (torch.zeros(tokens, cols, dtype=dtype, device=DEV) for _ in range(4))
        self.mean, self.rstd, self.losses = (torch.zeros(tokens, device=DEV) for _ in range(3))
        self.loss, self.count = torch.zeros(1, device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV)
        self.ids, self.labels = (torch.zeros(tokens, dtype=torch.int64, device=DEV) for _ in range(2))

    def text(self, seed):
        """Another text: the next word is the label, and a tenth of the positions do not count."""
        gen = torch.Generator(DEV).manual_seed(1000 + seed)
        words = torch.randint(0, self.vocab, (self.tokens + 1,), generator=gen, device=DEV)
        words[self.tokens // 2:self.tokens // 2 + 40] = 7  # a run of one word
        self.ids.copy_(words[:-1])
        self.labels.copy_(words[1:])
        self.labels[torch.rand(self.tokens, generator=gen, device=DEV) < 0.1] = -100

    def gradients(self):
        self.embedding.forward(self.ids, self.x)
        self.norm.forward(self.x, self.h, self.mean, self.rstd)
        self.head.grad(self.h, self.labels, self.losses, self.loss, self.count, self.dh, self.grads[0],
                       step_state=self.decision.state)
        self.norm.grad(self.x, self.dh, self.mean, self.rstd, self.dx, self.grads[1], self.grads[2])
        self.embedding.grad(self.ids, self.dx, self.grads[0], accumulate=True)  # the table is the head

    def step(self):
        self.gradients()
        self.decision.step()

    def reference(self):
        """Loss and gradients in 64 bits, from the parameters as they are."""
        table, weight, bias = (p.double().requires_grad_() for p in self.params)
        x = table[self.ids] * self.scale
        x = x - x.mean(1, keepdim=True)
        h = x * (x.square().mean(1, keepdim=True) + 1e-5).rsqrt() * weight + bias
        z = h @ table.t()
        counts = self.labels >= 0
        label = self.labels.clamp(min=0)[:, None]
        losses = torch.logsumexp(z, 1) - z.gather(1, label)[:, 0]
        loss = losses[counts].mean()
        loss.backward()
        return loss.item(), [p.grad for p in (table, weight, bias)]

    def everything(self):
        return [*self.params, *self.grads, *(t for x in self.state.values() for t in x), self.losses, self.loss,
                self.count, self.dh, self.dx, self.x, self.h]


@pytest.mark.parametrize("dtype,loss_scale", [(torch.bfloat16, 1.0), (torch.float16, 512.0)])
@pytest.mark.parametrize("vocab,cols,tokens", [(300, 64, 200), (1009, 136, 700)])
def test_steps_against_64_bits(dtype, loss_scale, vocab, cols, tokens):
    """Between the parameters and a gradient lie at most seven roundings to 16 bits (x, h, the factor, dh, dx, and dW
    twice), each off by eps / 2 of its value at most; what those of x and h change in the scores adds as much again at
    these widths: 8 eps of the gradient's 2-norm.  The update is checked on the gradients as they are."""
    model = Model(dtype, vocab, cols, tokens, loss_scale)
    bound = 8 * torch.finfo(dtype).eps
    for it in range(3):
        model.text(it)
        want_loss, want = model.reference()
        before = [[t.double() for t in x] for x in (model.state["master"], model.state["m"], model.state["v"])]
        model.step()
        torch.cuda.synchronize()
        assert abs(model.loss.item() - want_loss) <= bound * abs(want_loss)
        assert model.count.item() == int((model.labels >= 0).sum())
        for name, g, w in zip(("table", "weight", "bias"), model.grads, want):
            off = (g.double() / loss_scale - w).norm().item()
            assert off <= bound * w.norm().item(), (it, name, off / w.norm().item())
        decided = model.decision.read()
        norm = math.sqrt(sum(g.double().square().sum().item() for g in model.grads)) / loss_scale
        assert decided["skip"] == 0 and abs(decided["global_norm"] - norm) <= 1e-9 * norm
        c, t = model.config, it + 1
        factor = min(1.0, c.max_norm / (norm + 1e-6)) / loss_scale
        for k, g in enumerate(model.grads):
            p, m, v = (x[k] for x in before)
            g = g.double().view(-1) * factor
            m = c.beta1 * m + (1 - c.beta1) * g
            v = c.beta2 * v + (1 - c.beta2) * g * g
            p = p * (1 - c.lr * c.weight_decay) - c.lr / (1 - c.beta1**t) * m / (
                (v / (1 - c.beta2**t)).sqrt() + c.eps)
            # single roundings of p and of a step of at most about lr
            off = (model.state["master"][k].double() - p).abs().max().item()
            assert off <= 2.0**-22 * (p.abs().max().item() + c.lr), (it, k, off)
            assert torch.equal(model.params[k].view(-1), model.state["master"][k].to(dtype))


@pytest.mark.parametrize("dtype,loss_scale", [(torch.bfloat16, 1.0), (torch.float16, 64.0)])
def test_captured_steps_equal_eager_ones(dtype, loss_scale):
    """A captured step replayed on other texts, between eager work, against a twin's eager steps, bit for bit; the loss
    scale grows on the way, and the replays follow it."""
    a, b = (Model(dtype, 401, 72, 600, loss_scale, growth_interval=2, seed=5) for _ in range(2))
    for model in (a, b):
        model.text(9)
        model.step()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        a.step()
    for it in range(5):
        for model in (a, b):
            model.text(it)
        graph.replay()
        b.step()
        torch.randn(1000, device=DEV).sum()
        torch.cuda.synchronize()
        for k, (x, y) in enumerate(zip(a.everything(), b.everything())):
            assert torch.equal(x, y), (it, k)
    assert a.decision.read()["loss_scale"] == b.decision.read()["loss_scale"] == loss_scale * 8
    assert a.decision.read()["adam_step"] == 6


def test_a_loss_scale_that_overflows_skips_the_step():
    model = Model(torch.float16, 300, 64, 200, loss_scale=2.0**40)
    model.text(0)
    start = [p.clone() for p in model.params]
    skipped = 0
    for _ in range(40):
        model.step()
        if not model.decision.read()["skip"]:
            break
        skipped += 1
        assert all(torch.equal(p, q) for p, q in zip(model.params, start))
        assert model.loss.isfinite().all()
    decided = model.decision.read()
    assert 0 < skipped < 40 and decided["adam_step"] == 1 and decided["loss_scale"] == 2.0 ** (40 - skipped)
    assert not torch.equal(model.params[0], start[0])


def test_two_streams_with_operators_of_their_own():
    """Two models train at the same time on two streams as they do one after the other."""
    models = [Model(torch.bfloat16, 500, 128, 700, seed=s) for s in (1, 2)]
    alone = [Model(torch.bfloat16, 500, 128, 700, seed=s) for s in (1, 2)]
    for model in models + alone:
        model.text(9)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in models]
    for _ in range(3):
        for model, stream in zip(models, streams):
            with torch.cuda.stream(stream):
                model.step()
    torch.cuda.synchronize()
    for model, twin in zip(models, alone):
        for _ in range(3):
            twin.step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(model.everything(), twin.everything()))


def test_operators_that_share_a_workspace():
    """Operators whose calls follow one another on one stream may share a workspace: none relies on what is in it."""
    a, b = (Model(torch.bfloat16, 500, 128, 700, seed=3) for _ in range(2))
    room = b.head.ws
    b.embedding = TokenEmbedding(b.params[0], max_tokens=700, scale=b.scale, workspace=room)
    b.norm = LayerNorm(b.params[1], b.params[2], workspace=room)
    for model in (a, b):
        model.text(1)
        for _ in range(2):
            model.step()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a.everything(), b.everything()))


def test_calls_on_a_given_stream_and_fewer_tokens():
    """A stream as an argument, and a call of fewer tokens than the operators were made for."""
    a, b = (Model(torch.bfloat16, 300, 64, n, seed=4) for n in (1500, 600))
    b.text(2)
    a.ids[:600], a.labels[:600] = b.ids, b.labels
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    a.embedding.forward(a.ids[:600], a.x[:600], stream=s)
    a.norm.forward(a.x[:600], a.h[:600], a.mean[:600], a.rstd[:600], stream=s)
    a.head.grad(a.h[:600], a.labels[:600], a.losses[:600], a.loss, a.count, a.dh[:600], a.grads[0], stream=s)
    a.norm.grad(a.x[:600], a.dh[:600], a.mean[:600], a.rstd[:600], a.dx[:600], a.grads[1], a.grads[2],
                stream=s.cuda_stream)
    a.embedding.grad(a.ids[:600], a.dx[:600], a.grads[0], accumulate=True, stream=s)
    b.gradients()
    torch.cuda.synchronize()
    for x, y in ((a.loss, b.loss), (a.losses[:600], b.losses), (a.dx[:600], b.dx), *zip(a.grads, b.grads)):
        assert torch.equal(x, y)
    assert not a.x[600:].any() and not a.losses[600:].any()  # rows behind the last one are left as they were


def test_refusals():
    m = Model(torch.bfloat16, 300, 64, 200)
    far = torch.zeros(201, 64, dtype=torch.bfloat16, device=DEV)
    ids = torch.zeros(201, dtype=torch.int64, device=DEV)
    before = [t.clone() for t in m.everything()]
    with pytest.raises(ValueError, match="max_tokens"):
        m.embedding.grad(ids, far, m.grads[0])
    with pytest.raises(ValueError, match="max_tokens"):
        m.head.forward(far, ids, torch.zeros(201, device=DEV), m.loss, m.count)
    with pytest.raises(ValueError, match="max_tokens"):
        TokenEmbedding(m.params[0]).grad(m.ids, m.dx, m.grads[0])
    with pytest.raises(ValueError, match="without gradients"):
        LossHead(m.params[0], max_tokens=200, gradients=False).grad(m.h, m.labels, m.losses, m.loss, m.count, m.dh,
                                                                   m.grads[0])
    with pytest.raises(ValueError, match="a tensor on cpu"):
        m.embedding.forward(m.ids.cpu(), m.x)
    with pytest.raises(ValueError, match="a tensor on cpu"):
        m.norm.forward(m.x, m.h.cpu())
    with pytest.raises(ValueError, match="a tensor on cpu"):
        m.head.forward(m.h, m.labels, m.losses.cpu(), m.loss, m.count)
    with pytest.raises(ValueError, match="199 tokens for 200 rows"):
        m.embedding.forward(m.ids[:199], m.x)
    with pytest.raises(ValueError, match="gradient of"):
        m.embedding.grad(m.ids, m.dx, m.grads[0][:299])
    with pytest.raises(ValueError, match="int32 or int64"):
        m.embedding.forward(m.ids.float(), m.x)
    with pytest.raises(ValueError, match="contiguous tensor"):
        m.embedding.forward(torch.zeros(400, dtype=torch.int64, device=DEV)[::2], m.x)
    with pytest.raises(ValueError, match="rows must be contiguous"):
        m.norm.forward(torch.zeros(64, 200, dtype=torch.bfloat16, device=DEV).t(), m.h)
    with pytest.raises(ValueError, match="overlap"):
        m.norm.grad(m.x, m.dh, m.mean, m.rstd, torch.zeros(1, 64, dtype=torch.bfloat16, device=DEV).expand(200, 64))
    with pytest.raises(ValueError, match="mean"):
        m.norm.forward(m.x, m.h, m.mean.double(), m.rstd)
    with pytest.raises(Z.ZeroError, match="statistics"):
        m.norm.grad(m.x, m.dh, None, m.rstd, m.dx)
    with pytest.raises(Z.ZeroError, match="another shape or dtype"):
        m.norm.forward(m.x, torch.zeros(200, 64, device=DEV))
    with pytest.raises(Z.ZeroError, match="16-bit"):
        m.head.forward(m.h.float(), m.labels, m.losses, m.loss, m.count)
    with pytest.raises(Z.ZeroError, match="differ in cols"):
        m.head.forward(torch.zeros(200, 72, dtype=torch.bfloat16, device=DEV), m.labels, m.losses, m.loss, m.count)
    with pytest.raises(Z.ZeroError, match="scale"):
        m.head.grad(m.h, m.labels, m.losses, m.loss, m.count, m.dh, m.grads[0], scale=math.inf)
    with pytest.raises(ValueError, match="a workspace of"):
        LossHead(m.params[0], max_tokens=200, workspace=torch.zeros(10, dtype=torch.uint8, device=DEV))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(before, m.everything()))


def far_rows(x, stride=2**30 + 8):
    """The rows of x so far apart that the third begins past 2^32 bytes."""
    out = torch.empty((x.shape[0] - 1) * stride + x.shape[1], dtype=x.dtype, device=DEV)
    out = out.as_strided(x.shape, (stride, 1))
    out.copy_(x)
    return out


def test_offsets_past_32_bits():
    gen = torch.Generator(DEV).manual_seed(8)
    near = [torch.randn(3, 64, generator=gen, device=DEV).bfloat16() for _ in range(6)]
    far = [far_rows(t) for t in near]
    weight = torch.randn(64, generator=gen, device=DEV).bfloat16()
    results = []
    for table, x, dy, out, dx, dw in (near, far):
        for tokens in (300, 700):  # both ways of the table's gradient
            ids = torch.arange(tokens, device=DEV) % 4 - 1  # one in four names no row
            many = torch.randn(tokens, 64, generator=torch.Generator(DEV).manual_seed(1), device=DEV).bfloat16()
            op = TokenEmbedding(table, max_tokens=tokens)
            op.grad(ids, many, dw)
            results.append(dw.clone())
            op.forward(ids, many)
            results.append(many.clone())
        op.forward(torch.tensor([2, 0, 1], device=DEV), out)
        results.append(out.clone())
        norm, mean, rstd = LayerNorm(weight, weight), torch.zeros(3, device=DEV), torch.zeros(3, device=DEV)
        norm.forward(x, out, mean, rstd)
        results += [out.clone(), mean, rstd]
        wg = torch.zeros(64, device=DEV)
        norm.grad(x, dy, mean, rstd, dx, wg)
        results += [dx.clone(), wg]
        head = LossHead(table, max_tokens=3)
        losses, loss, count = torch.zeros(3, device=DEV), torch.zeros(1, device=DEV), torch.zeros(
            1, dtype=torch.int64, device=DEV)
        head.grad(x, torch.tensor([2, 1, 0], device=DEV), losses, loss, count, dx, dw)
        results += [losses, loss, count, dx.clone(), dw.clone()]
    torch.cuda.synchronize()
    half = len(results) // 2
    assert all(torch.equal(a, b) for a, b in zip(results[:half], results[half:]))
