"""Lists past 32-bit indices: one tensor of 2^32 + 5003 elements and a small one behind it, over many launches.  Inputs
repeat with a period of 2^20 + 7 elements, so windows anywhere are known without holding the whole."""
import numpy as np
import pytest
import torch

from tests import list_reference as R
from tests import parity

pytestmark = [pytest.mark.gpu, pytest.mark.slow]

if torch.cuda.is_available():
    import mixed_precision_adam_amd as Z
    from mixed_precision_adam_amd.driver import TensorList

DEV = "cuda:0"
N, SMALL, PERIOD = 2**32 + 5003, 1000, 2**20 + 7
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)
WINDOWS = [(0, 4096), (2**25 - 4096, 2**25 + 4096), (2**31 - 4096, 2**31 + 4096), (2**32 - 4096, 2**32 + 4096),
           ((N - 8192) // 4096 * 4096, N)]


def repeated(period, out):
    """`period` over and over, in pieces."""
    for lo in range(0, out.numel(), PERIOD * 64):
        piece = out[lo:lo + PERIOD * 64]
        piece.copy_(period.repeat(64)[:piece.numel()])
    return out


@pytest.fixture(scope="module")
def inputs():
    if torch.cuda.get_device_properties(0).total_memory < 200 * 2**30:
        pytest.skip("needs 200 GiB of device memory")
    rng = np.random.default_rng(3)
    host = torch.from_numpy((rng.standard_normal(PERIOD) * 1e-3).astype(np.float32)).bfloat16()
    grad = repeated(host.to(DEV), torch.empty(N, dtype=torch.bfloat16, device=DEV))
    yield host.float().numpy(), grad
    del grad
    torch.cuda.empty_cache()


def at(period, lo, hi):
    return period[np.arange(lo, hi) % PERIOD]


def test_norm(inputs):
    g, grad = inputs
    small = torch.full((SMALL,), 0.5, device=DEV)
    out = torch.zeros(2, dtype=torch.float64, device=DEV)
    flag = out[1:].view(torch.int32)
    lst = TensorList([N, SMALL], [grad, small])
    lst.grad_sqnorm(out[:1], flag)
    sq = g.astype(np.float64) ** 2
    want = (N // PERIOD) * np.sum(sq.astype(np.longdouble)) + np.sum(sq[:N % PERIOD].astype(np.longdouble)) + 250.0
    assert abs(float(out[0]) - float(want)) <= N * 2.0**-53 * float(want) and int(flag[0]) == 0
    grad[N - 1] = float("nan")
    lst.grad_sqnorm(out[:1], flag)
    assert int(flag[0]) == 1
    grad[N - 1] = float(at(g, N - 1, N)[0])


def test_adamw(inputs):
    g, grad = inputs
    state = [torch.zeros(Z.zero_state_tiled_numel(n), device=DEV) for n in (N, SMALL)]
    param = [torch.zeros(n, dtype=torch.bfloat16, device=DEV) for n in (N, SMALL)]
    small = torch.full((SMALL,), 0.5, device=DEV)
    TensorList([N, SMALL], [grad, small], param, state=state).adamw(Z.zero_list_hparams([dict(HP, step=1)]))
    s = R.scalars(**HP, grad_scale=1.0, step=1)
    for k, lo, hi in [(0, a, b) for a, b in WINDOWS] + [(1, 0, SMALL)]:
        x = at(g, lo, hi) if k == 0 else np.full(SMALL, 0.5, np.float32)
        want = R.adamw(x, *(np.zeros(hi - lo, np.float32),) * 3, s)
        tiles = state[k].view(-1, 3, 1024)[lo // 1024:-(-hi // 1024)].cpu().numpy()
        for name, j in (("master", 0), ("m", 1), ("v", 2)):
            parity.assert_bits_equal(tiles[:, j].reshape(-1)[:hi - lo], want[j], f"{name} {lo}")
        got = param[k][lo:hi].cpu().view(torch.int16).numpy()
        parity.assert_bits_equal(got, torch.from_numpy(want[0]).bfloat16().view(torch.int16).numpy(), f"param {lo}")


def test_adamw8_and_unpack(inputs):
    g, grad = inputs
    state = [torch.zeros(Z.zero_state8_bytes(n), dtype=torch.uint8, device=DEV) for n in (N, SMALL)]
    param = [torch.zeros(n, dtype=torch.bfloat16, device=DEV) for n in (N, SMALL)]
    small = torch.full((SMALL,), 0.5, device=DEV)
    lst = TensorList([N, SMALL], [grad, small], param, state8=state)
    lst.adamw(Z.zero_list_hparams([dict(HP, step=1)]), seed=5)
    back = {k: [torch.zeros(n, device=DEV) for n in (N, SMALL)] for k in ("master", "m", "v")}
    lst.unpack8(TensorList([N, SMALL], **back))
    s = R.scalars(**HP, grad_scale=1.0, step=1)
    for k, lo, hi in [(0, a, b) for a, b in WINDOWS] + [(1, 0, SMALL)]:
        x = at(g, lo, hi) if k == 0 else np.full(SMALL, 0.5, np.float32)
        raw = state[k].view(-1, 24704)[lo // 4096:-(-hi // 4096)].reshape(-1).cpu().numpy()
        st = R.State8(raw, hi - lo)
        zero = R.State8(np.zeros_like(raw), hi - lo)
        block0 = lo // 256 if k == 0 else -(-N // 4096) * 16
        _, cm, cv, sm, sv = R.adamw8(x, zero, s, 5, 1, block0)
        n = hi - lo
        for name, a, b in (("m", st.m.reshape(-1)[:n], cm.reshape(-1)[:n]), ("v", st.v.reshape(-1)[:n],
                                                                             cv.reshape(-1)[:n]),
                           ("m scale", st.scale_m, sm), ("v scale", st.scale_v, sv)):
            parity.assert_bits_equal(a, b, f"{name} {lo}")
        m, v = st.moments()
        for name, want in (("master", st.master), ("m", m), ("v", v)):
            parity.assert_bits_equal(back[name][k][lo:hi].cpu().numpy(), want, f"unpacked {name} {lo}")
