"""One AdamWConfig gives the flat step and the step over lists the same decision, on the GPU."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mixed_precision_adam_amd as Z
    from mixed_precision_adam_amd.driver import AdamWConfig, DeviceDecision, ListDecision, RankShard, TensorList

DEV = "cuda:0"


class Both:
    """The same gradients and parameters in a flat shard and in a list."""

    def __init__(self, cfg):
        numels = [5000, 17, 40_003]
        rng = np.random.default_rng(0)
        srcs = [torch.from_numpy(rng.standard_normal(n).astype(np.float32)).bfloat16().to(DEV) for n in numels]
        shard = RankShard(numels, 1, 0, Z.ZERO_BF16, DEV, sources=srcs, tiled=True, fused=True)
        shard.load_master(torch.zeros(shard.n, device=DEV))
        state = {k: [torch.zeros(n, device=DEV) for n in numels] for k in ("master", "m", "v")}
        params = [torch.zeros(n, dtype=torch.bfloat16, device=DEV) for n in numels]
        self.flat = DeviceDecision([shard], cfg)
        self.list = ListDecision(TensorList(numels, srcs, params, **state), [cfg])

    def step(self):
        """Both decisions; norms are summed in different orders: n·2^-53 of each, far below 1e-10."""
        self.flat.step()
        self.list.step()
        got, want = self.list.read(), self.flat.read()
        assert got["adam_step"] == want["adam_step"]
        for k in ("global_norm", "grad_scale"):
            assert got[k] == pytest.approx(want[k], rel=1e-10)
        assert got["scalars"][:8] == want["scalars"][:8]
        return got


@pytest.mark.parametrize("max_norm", [0.0, 0.1, 2.0])
def test_clipping(max_norm):
    both = Both(AdamWConfig(max_norm=max_norm))
    for _ in range(2):
        got = both.step()
        assert (got["grad_scale"] == 1.0) == (max_norm == 0.0)


def test_a_schedule():
    """lr and max_norm set between steps."""
    cfg = AdamWConfig(lr=1e-3)
    both = Both(cfg)
    for lr, norm in ((1e-3, 1.0), (5e-4, 1.0), (2e-4, 0.5)):
        cfg.lr, cfg.max_norm = lr, norm
        got = both.step()
        step, t = got["scalars"][6], got["adam_step"]
        assert step == pytest.approx(lr / (1 - 0.9**t), rel=1e-6)  # one rounding to fp32: 2^-24
