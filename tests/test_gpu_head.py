"""The loss head (softmax cross entropy over a large vocabulary) against a plain implementation in 64 bits, on the GPU.

Tolerances.  A score is a sum of d products in fp32: off by at most d * 2^-24 of the sum of their magnitudes, S.  Losses
are two such scores apart and add a handful of roundings of the largest.  A factor of the gradients' products (softmax -
onehot) comes from a score held to 2^-12 of an octave and is rounded once to 16 bits: off by e = 2^-12 ln 2 + eps / 2
of itself, and by what the scores are off; a word further than 32 octaves below its piece's maximum counts as 0."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_ends import DEV, U, between, check, half_step, matrix

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mixed_precision_adam_amd as Z
    from mixed_precision_adam_amd.driver import LossHead

FORMATS = {"bf16": torch.bfloat16, "fp16": torch.float16}


class Head:
    """Inputs of one call, its outputs (with what lies between their rows), and the results in 64 bits."""

    def __init__(self, tokens, vocab, cols, dt, spare=0, shift=0, ignored=0.2, seed=0, sigma=0.05, sure=0.0):
        gen = torch.Generator(DEV).manual_seed(tokens * 7 + vocab * 3 + cols + seed)
        self.dtype = FORMATS[dt]
        self.table, _ = matrix(vocab, cols, self.dtype, gen, sigma, spare, shift)
        self.labels = torch.randint(0, vocab, (tokens,), generator=gen, device=DEV)
        self.x, _ = matrix(tokens, cols, self.dtype, gen, 1.0, spare, shift)
        if sure:
            self.x.add_((self.table[self.labels].float() * (sure / (sigma * sigma * cols))).to(self.dtype))
        self.labels[torch.rand(tokens, generator=gen, device=DEV) < ignored] = -100
        self.losses = torch.full((tokens,), 9.0, device=DEV)
        self.loss, self.count = torch.full((1,), 9.0, device=DEV), torch.full((1,), 9, device=DEV)
        self.dx, self.dx_buf = matrix(tokens, cols, self.dtype, gen, 1.0, spare, shift)
        self.dw, self.dw_buf = matrix(vocab, cols, self.dtype, gen, 0.01, spare, shift)
        self.old = self.dw.clone()
        self.rest = between(self.dx, self.dx_buf), between(self.dw, self.dw_buf)
        self.vocab, self.cols = vocab, cols

    def want(self, scale=1.0):
        x, w = self.x.double(), self.table.double()
        counts = (self.labels >= 0) & (self.labels < self.vocab)
        x = torch.where(counts[:, None], x, 0.0)
        label = self.labels.clamp(0, self.vocab - 1)[:, None]
        z = x @ w.t()
        slack_z = self.cols * U * (x.abs() @ w.abs().t())  # of each score
        lse = torch.logsumexp(z, 1, keepdim=True)
        slack = slack_z.amax(1, keepdim=True) + 16 * U * (1 + z.abs().amax(1, keepdim=True))
        self.counts = counts
        self.want_losses = torch.where(counts, (lse - z.gather(1, label))[:, 0], 0.0)
        self.slack_losses = 2 * slack[:, 0]
        n = max(1, int(counts.sum()))
        factor = scale / n
        p = (z - lse).exp()
        g = p.scatter_add(1, label, torch.full_like(lse, -1.0))
        g.scatter_(1, label, torch.expm1(-self.want_losses)[:, None])
        fmt = torch.finfo(self.dtype)
        least = fmt.tiny * fmt.eps / (2 if self.dtype == torch.bfloat16 else 2.0**16)  # half the least step of a factor
        e = g.abs() * (2.0**-12 * math.log(2) + fmt.eps / 2) + (p + g.abs()) * 2 * slack + 2.0**-31 + least
        g, e = g * counts[:, None], e * counts[:, None]
        self.want_dx, self.slack_dx = (g @ w) * factor, (e @ w.abs()) * factor
        self.slack_dx += 2.0**-14 * self.slack_dx + self.vocab * U * (g.abs() @ w.abs()) * factor
        self.want_dw, self.slack_dw = (g.t() @ x) * factor, (e.t() @ x.abs()) * factor
        self.slack_dw += len(x) * U * (g.abs().t() @ x.abs()) * factor
        return self

    def check_losses(self):
        check("losses", self.losses, self.want_losses, self.slack_losses + U * self.want_losses.abs())
        n = int(self.counts.sum())
        assert self.count.item() == n
        check("loss", self.loss, self.want_losses.sum().view(1) / max(1, n),
              self.slack_losses.max().view(1) + U * self.want_losses.abs().max() if n else torch.zeros(1, device=DEV))

    def check_grads(self, accumulate):
        check("x_grad", self.dx, self.want_dx, half_step(self.want_dx, self.dtype) * 1.01 + self.slack_dx)
        want = self.want_dw + (self.old.double() if accumulate else 0.0)
        check("table_grad", self.dw, want, half_step(want, self.dtype) * 1.01 + self.slack_dw + U * want.abs())
        assert torch.equal(between(self.dx, self.dx_buf), self.rest[0])
        assert torch.equal(between(self.dw, self.dw_buf), self.rest[1])

    def outputs(self):
        return [self.losses, self.loss, self.count, self.dx, self.dw]


SIZES = [(1, 1, 1, 0, 0), (1, 300, 64, 0, 0), (3, 257, 40, 0, 0), (33, 1000, 129, 3, 1), (256, 512, 64, 8, 0),
         (257, 255, 192, 0, 0), (300, 4099, 72, 1, 0), (700, 777, 1600, 0, 8), (64, 20_011, 264, 0, 0)]


@pytest.mark.parametrize("dt", FORMATS)
@pytest.mark.parametrize("tokens,vocab,cols,spare,shift", SIZES)
def test_losses(tokens, vocab, cols, spare, shift, dt):
    h = Head(tokens, vocab, cols, dt, spare, shift).want()
    op = LossHead(h.table, max_tokens=tokens, gradients=False)
    op.ws.fill_(0xFF)
    op.forward(h.x, h.labels.int(), h.losses, h.loss, h.count)
    h.check_losses()


@pytest.mark.parametrize("dt", FORMATS)
@pytest.mark.parametrize("tokens,vocab,cols,spare,shift", SIZES)
def test_gradients(tokens, vocab, cols, spare, shift, dt):
    state = torch.zeros(16, dtype=torch.float64, device=DEV)
    Z.zero_step_state_init(state, 64.0, 1000)
    for accumulate, sure in ((False, 0.0), (True, 12.0)):
        h = Head(tokens, vocab, cols, dt, spare, shift, seed=int(sure), sure=sure)
        with_state = dt == "fp16"
        h.want(0.5 * (64.0 if with_state else 1.0))
        op = LossHead(h.table, max_tokens=tokens + 300)
        op.ws.fill_(0xFF)  # NaN wherever something is taken that nobody wrote
        op.grad(h.x, h.labels, h.losses, h.loss, h.count, h.dx, h.dw, accumulate=accumulate,
                step_state=state if with_state else None, scale=0.5)
        h.check_losses()
        h.check_grads(accumulate)
        first = [t.clone() for t in h.outputs()]
        h.dw.copy_(h.old)
        op.grad(h.x, h.labels.int(), h.losses, h.loss, h.count, h.dx, h.dw, accumulate=accumulate,
                step_state=state if with_state else None, scale=0.5)
        assert all(torch.equal(a, b) for a, b in zip(first, h.outputs()))


@pytest.mark.parametrize("accumulate", [False, True])
def test_more_tokens_than_one_block_holds(accumulate):
    """A vocabulary of 2^18 + 1 words leaves blocks of 256 tokens: three of them, the last with one token."""
    h = Head(513, (1 << 18) + 1, 24, "bf16", ignored=0.1).want(2.0)
    op = LossHead(h.table, max_tokens=513)
    op.ws.fill_(0xFF)
    op.grad(h.x, h.labels, h.losses, h.loss, h.count, h.dx, h.dw, accumulate=accumulate, scale=2.0)
    h.check_losses()
    h.check_grads(accumulate)


@pytest.mark.parametrize("dt", FORMATS)
def test_no_token_counts(dt):
    """All labels outside the vocabulary, and no tokens at all: losses and gradients of zeros, or nothing added."""
    for tokens in (0, 5, 300):
        h = Head(max(tokens, 1), 100, 64, dt)
        x, losses, dx = h.x[:tokens], h.losses[:tokens], h.dx[:tokens]
        x.fill_(float("nan"))  # their rows have no part in the gradients, whatever they hold
        labels = torch.tensor([-1, 100, 2**40, -2**40, -100] * 60, device=DEV)[:tokens]
        op = LossHead(h.table, max_tokens=tokens)
        op.grad(x, labels, losses, h.loss, h.count, dx, h.dw, accumulate=True)
        assert torch.equal(h.dw, h.old) and not dx.any() and not losses.any()
        assert h.loss.item() == 0.0 and h.count.item() == 0
        op.grad(x, labels, losses, h.loss, h.count, dx, h.dw)
        assert not h.dw.any()


def test_rows_that_do_not_count_may_hold_anything():
    h = Head(290, 500, 136, "bf16", ignored=0.4)
    h.x[h.labels < 0] = float("inf")
    h.x[(h.labels < 0).nonzero()[:3, 0]] = float("nan")
    h.want()
    LossHead(h.table, max_tokens=290).grad(h.x, h.labels, h.losses, h.loss, h.count, h.dx, h.dw)
    h.check_losses()
    h.check_grads(False)


def test_scores_that_are_not_finite():
    """A word at -inf has probability 0; +inf and NaN make their token NaN and leave the others alone."""
    h = Head(40, 300, 64, "bf16", ignored=0.0)
    with torch.no_grad():
        h.x[:, 0] = 0.0
        h.x[3, 0] = float("nan")
        h.x[5, 0] = 1.0
        h.table[:, 0] = 0.0
        h.table[7, 0] = float("-inf")  # 0 * inf is NaN: seen by every token
    h.labels[:] = 9
    op = LossHead(h.table, max_tokens=40)
    op.forward(h.x, h.labels, h.losses, h.loss, h.count)
    bad = h.losses.isnan()
    assert bad[[0, 1, 3]].all()  # 0 * -inf
    assert not bad[5]  # 1 * -inf = -inf
    z = h.x[5].double() @ h.table.double().t()
    assert abs(h.losses[5].item() - (torch.logsumexp(z, 0) - z[9]).item()) < 1e-4
    h.table[7, 0] = 0.0
    h.x[3, 0] = 1.0
    h.x[8] = float("nan")
    op.grad(h.x, h.labels, h.losses, h.loss, h.count, h.dx, h.dw)
    bad = h.losses.isnan()
    assert bad.nonzero()[:, 0].tolist() == [8] and h.loss.isnan()
    assert h.dx[8].isnan().all() and h.dx[torch.arange(40, device=DEV) != 8].isfinite().all()
    assert h.dw.isnan().all()


def test_scores_far_apart():
    """Scores over hundreds of octaves: no overflow, no loss of the words near the maximum."""
    h = Head(70, 700, 64, "bf16", sigma=4.0, ignored=0.0).want()
    LossHead(h.table, max_tokens=70).grad(h.x, h.labels, h.losses, h.loss, h.count, h.dx, h.dw)
    h.check_losses()
    h.check_grads(False)


def test_gradients_against_differences():
    """Central differences of the loss in 64 bits; the factors are off by 2^-9 of themselves, so the sums by 2^-8 of
    the largest gradient at most."""
    h = Head(6, 40, 16, "fp16", ignored=0.0, sigma=0.3).want()
    LossHead(h.table, max_tokens=6).grad(h.x, h.labels, h.losses, h.loss, h.count, h.dx, h.dw)

    def loss(x, w):
        z = x @ w.t()
        return (torch.logsumexp(z, 1) - z.gather(1, h.labels[:, None])[:, 0]).mean().item()

    point, step = [h.x.double(), h.table.double()], 1e-5
    for k, grad in enumerate((h.dx, h.dw)):
        for i in range(0, point[k].numel(), 11):
            found = []
            for sign in (1, -1):
                moved = [p.clone() for p in point]
                moved[k].view(-1)[i] += sign * step
                found.append(loss(*moved))
            want = (found[0] - found[1]) / (2 * step)
            assert abs(grad.reshape(-1)[i].item() - want) <= 2.0**-8 * grad.abs().max().item(), (k, i)


@pytest.mark.parametrize("accumulate", [False, True])
def test_more_tokens_than_one_block_holds_over_a_small_vocabulary(accumulate):
    """Rows of 16384 columns leave blocks of 8192 tokens whatever the vocabulary: two of them, the second ragged."""
    h = Head(8192 + 259, 40, 16384, "bf16", ignored=0.1, sigma=5e-4).want(2.0)
    op = LossHead(h.table, max_tokens=8192 + 259)
    op.ws.fill_(0xFF)
    op.grad(h.x, h.labels, h.losses, h.loss, h.count, h.dx, h.dw, accumulate=accumulate, scale=2.0)
    h.check_losses()
    h.check_grads(accumulate)


@pytest.mark.parametrize("dt", FORMATS)
@pytest.mark.parametrize("high", [24.0, 40.0, -40.0])
def test_tokens_that_are_sure_of_their_word(dt, high):
    """Scores that fp32 holds exactly: `high` for the label, half of it for the 99 others (the label's loss is
    log(1 + 99 e^(-high / 2)), 2e-7 at 40).  In octaves the two scores are off by 1.5 * 2^-24 of themselves, their
    difference by 1.5 * 2^-24 * 1.5 * |high| log2(e) = 3.3 |high| 2^-24; the logarithm of the others' sum, its addition
    and the difference round once at 2 |high| 2^-24 at most together, so the loss is off by less than
    8 |high| 2^-24 of itself where it is small, and by that many octaves where it is large.  A factor is off by one
    rounding of its format and by as much as the loss."""
    n, vocab = 70, 100
    dtype = FORMATS[dt]
    x, table = (torch.zeros(k, 64, dtype=dtype, device=DEV) for k in (n, vocab))
    x[:, 0], table[:, 0], table[9, 0] = abs(high), math.copysign(0.5, high), math.copysign(1.0, high)
    labels = torch.full((n,), 9, device=DEV)
    losses, loss = torch.zeros(n, device=DEV), torch.zeros(1, device=DEV)
    count = torch.zeros(1, dtype=torch.int64, device=DEV)
    dx, dw = torch.zeros_like(x), torch.zeros_like(table)
    scale = 2.0**17 if high > 30 else 1.0  # keeps the gradients among the format's normal numbers
    LossHead(table, max_tokens=n).grad(x, labels, losses, loss, count, dx, dw, scale=scale)
    rest = math.log(99.0) - high / 2
    want = math.log1p(math.exp(rest)) if rest < 0 else rest + math.log1p(math.exp(-rest))
    off = 8 * abs(high) * U * max(want, 1.0 if want > 0.5 else want)
    assert (losses.double() - want).abs().max().item() <= off
    assert abs(loss.item() - want) <= off + 2 * U * want
    assert count.item() == n
    step = torch.finfo(dtype).eps / 2
    g = -math.expm1(-want) * scale / n  # of the label, negative; the others' factors add up to it
    rel = step + 2.0**-12 * math.log(2) + 8 * abs(high) * U
    want_dx = -g * math.copysign(0.5, high)
    assert (dx[:, 0].double() - want_dx).abs().max().item() <= 1.01 * abs(want_dx) * (3 * rel + step)
    assert not dx[:, 1:].any() and not dw[:, 1:].any()
    want_dw = torch.full((vocab,), g / 99 * n * abs(high), dtype=torch.float64, device=DEV)
    want_dw[9] = -g * n * abs(high)
    assert ((dw[:, 0].double() - want_dw).abs() <= 1.01 * want_dw.abs() * (rel + step)).all()


@pytest.mark.parametrize("gradients", [False, True])
@pytest.mark.parametrize("tokens,vocab,cols,spare", [(33, 300, 64, 0), (300, 777, 192, 8), (300, 777, 192, 3)])
def test_a_table_read_where_it_is_needs_no_room_for_a_copy(tokens, vocab, cols, spare, gradients):
    """The operator's workspace is what its table needs, and what lies behind it is left alone."""
    h = Head(tokens, vocab, cols, "bf16", spare).want()
    need = Z.zero_loss_head_workspace_bytes_for(tokens, h.table, gradients)
    copy = 0 if spare % 8 else -(-2 * vocab * cols // 256) * 256
    assert need == Z.zero_loss_head_workspace_bytes(tokens, vocab, cols, gradients) - copy
    assert LossHead(h.table, max_tokens=tokens, gradients=gradients).ws.numel() == need
    room = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device=DEV)
    op = LossHead(h.table, max_tokens=tokens, gradients=gradients, workspace=room)
    if gradients:
        op.grad(h.x, h.labels, h.losses, h.loss, h.count, h.dx, h.dw)
        h.check_grads(False)
    else:
        op.forward(h.x, h.labels, h.losses, h.loss, h.count)
    h.check_losses()
    assert (room[need:] == 0xFF).all()
    with pytest.raises(ValueError, match="16-bit"):
        LossHead(h.table.float(), max_tokens=tokens)


@pytest.mark.parametrize("tokens,vocab,cols", [(300, 777, 192), (513, (1 << 18) + 1, 24)])
def test_hidden_rows_may_be_overwritten_by_their_gradient(tokens, vocab, cols):
    """x_grad over x, in one block of tokens and in three: the bits of a call with memory of its own."""
    h = Head(tokens, vocab, cols, "bf16")
    op = LossHead(h.table, max_tokens=tokens)
    op.grad(h.x, h.labels, h.losses, h.loss, h.count, h.dx, h.dw)
    x, dw = h.x.clone(), torch.zeros_like(h.dw)
    op.grad(x, h.labels, h.losses, h.loss, h.count, x, dw)
    assert torch.equal(x, h.dx) and torch.equal(dw, h.dw)


@pytest.mark.parametrize("label,others,want", [
    (math.inf, 0.0, math.nan), (math.nan, 0.0, math.nan), (0.0, math.inf, math.nan), (0.0, math.nan, math.nan),
    (-math.inf, 0.0, math.inf), (0.0, -math.inf, 0.0), (-math.inf, -math.inf, math.nan),
    (-math.inf, math.inf, math.nan), (math.inf, -math.inf, math.nan), (1e30, 0.0, 0.0), (0.0, 1e30, 1e30)])
@pytest.mark.parametrize("vocab", [2, 64, 65, 300])
def test_losses_of_scores_at_the_ends_of_the_range(label, others, want, vocab):
    """One score for the label, one for all other words.  1e30 in bf16 is off by half a step of its own."""
    table = torch.zeros(vocab, 64, dtype=torch.bfloat16, device=DEV)
    table[:, 0], table[1, 0] = others, label
    x = torch.zeros(3, 64, dtype=torch.bfloat16, device=DEV)
    x[:, 0] = 1.0
    labels = torch.tensor([1, -1, 1], device=DEV)
    losses, loss = torch.full((3,), 9.0, device=DEV), torch.zeros(1, device=DEV)
    count = torch.zeros(1, dtype=torch.int64, device=DEV)
    dx, dw = torch.zeros_like(x), torch.zeros_like(table)
    op = LossHead(table, max_tokens=3)
    for call in (lambda: op.forward(x, labels, losses, loss, count),
                 lambda: op.grad(x, labels, losses, loss, count, dx, dw)):
        call()
        assert losses[1].item() == 0.0 and count.item() == 2
        for got in (losses[0].item(), losses[2].item(), loss.item()):
            assert got == pytest.approx(want, rel=2.0**-8, nan_ok=True), got
    assert not dx[1].any()
    if math.isnan(want):  # the token's factors, so its gradient and every word's
        assert dx[0, 0].isnan() and dw[:, 0].isnan().all()
    elif math.isfinite(label) and math.isfinite(others):
        sure = label > others
        assert torch.equal(dw[:, 0], torch.zeros_like(dw[:, 0])) if sure else dw[1, 0].item() == -1.0
