"""New gradients for a TensorList while its steps are queued elsewhere, on the GPU."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixed_precision_adam_amd.driver import AdamWConfig, ListDecision, TensorList

DEV = "cuda:0"
SIZES = [5, 70_001, 300_007]


class Model:
    """fp32 state, bf16 parameters and the gradients of the step `it`."""

    def __init__(self):
        rng = np.random.default_rng(1)
        self.state = {k: [torch.from_numpy((rng.standard_normal(n) * 1e-2).astype(np.float32)).abs_().to(DEV)
                          for n in SIZES] for k in ("master", "m", "v")}
        self.params = [torch.zeros(n, dtype=torch.bfloat16, device=DEV) for n in SIZES]
        self.list = TensorList(SIZES, self.grads(0), self.params, **self.state)
        self.run = ListDecision(self.list, [AdamWConfig(lr=1e-2)], max_norm=0.5)

    def grads(self, it):
        rng = np.random.default_rng(100 + it)
        return [torch.from_numpy((rng.standard_normal(n) * 1e-3).astype(np.float32)).to(DEV) for n in SIZES]

    def results(self):
        torch.cuda.synchronize()
        return [t.clone() for x in (*self.state.values(), self.params) for t in x]


def busy(stream, x):
    with torch.cuda.stream(stream):
        for _ in range(100):
            x.add_(1.0)


@pytest.mark.parametrize("captured", [False, True])
def test_new_gradients_behind_a_step_on_another_stream(captured):
    """Steps queued behind other work on a stream of their own take the gradients they were queued with, also when
    those are replaced, freed and their memory used again at once."""
    plain, x = Model(), Model()
    big = torch.zeros(1 << 28, device=DEV)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    if captured:
        with torch.cuda.graph(graph, stream=other):
            x.run.step()
    for it in range(3):
        if it:
            plain.list.set_grads(plain.grads(it))
        plain.run.step()
        torch.cuda.synchronize()
    for it in range(3):
        if it:
            x.list.set_grads(x.grads(it))
            junk = [torch.full((n,), 7.0, device=DEV) for n in SIZES for _ in range(4)]  # where freed gradients lay
        busy(other, big)
        if captured:
            with torch.cuda.stream(other):
                graph.replay()
        else:
            x.run.step(stream=other)
    for got, want in zip(x.results(), plain.results()):
        assert torch.equal(got, want)
    assert x.run.read()["adam_step"] == 3 and all((j == 7.0).all() for j in junk)
