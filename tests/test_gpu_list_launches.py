"""Conversion past one launch (2^26 elements): one tensor that ends in the second launch and a small one behind it.
Inputs repeat with a period of 2^20 + 7 elements, so windows anywhere are known without holding the whole."""
import numpy as np
import pytest
import torch

from tests import list_reference as R
from tests import parity

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mixed_precision_adam_amd as Z
    from mixed_precision_adam_amd.driver import TensorList

DEV = "cuda:0"
N, SMALL, PERIOD = 2**26 + 5003, 1000, 2**20 + 7
HALF = 1 << 19  # pack rounds to nearest
WINDOWS = [(0, 0, 8192), (0, 2**26 - 4096, N), (1, 0, SMALL)]


def repeated(period, n):
    return period.repeat(-(-n // PERIOD))[:n].clone()


@pytest.fixture(scope="module")
def packed():
    rng = np.random.default_rng(8)
    host = {"master": rng.standard_normal(PERIOD) * 0.02, "m": rng.standard_normal(PERIOD) * 3e-4,
            "v": rng.random(PERIOD) * 1e-6}
    host = {k: x.astype(np.float32) for k, x in host.items()}
    fp32 = {k: [repeated(torch.from_numpy(x).to(DEV), n) for n in (N, SMALL)] for k, x in host.items()}
    state = [torch.full((Z.zero_state8_bytes(n),), 9, dtype=torch.uint8, device=DEV) for n in (N, SMALL)]
    lst = TensorList([N, SMALL], state8=state)
    TensorList([N, SMALL], **fp32).pack8(lst)
    yield host, state, lst
    torch.cuda.empty_cache()


def window(host, lo, hi):
    return {k: x[np.arange(lo, hi) % PERIOD] for k, x in host.items()}


def test_pack(packed):
    host, state, _ = packed
    for k, lo, hi in WINDOWS:
        raw = state[k].view(-1, 24704)[lo // 4096:-(-hi // 4096)].reshape(-1).cpu().numpy()
        st, n, x = R.State8(raw, hi - lo), hi - lo, window(host, lo, hi)
        parity.assert_bits_equal(st.master, x["master"], f"master {k} {lo}")
        for name, codes, scale in (("m", st.m, st.scale_m), ("v", st.v, st.scale_v)):
            want, want_scale = R.encode(R.blocks_of(x[name]), name, HALF)
            parity.assert_bits_equal(codes.reshape(-1)[:n], want.reshape(-1)[:n], f"{name} codes {k} {lo}")
            parity.assert_bits_equal(scale, want_scale, f"{name} scales {k} {lo}")


@pytest.mark.parametrize("parts", [("m", "v"), ("master", "m", "v")])
def test_unpack(packed, parts):
    host, _, lst = packed
    back = {p: [torch.full((n + 16,), 3.0, device=DEV) for n in (N, SMALL)] for p in parts}
    lst.unpack8(TensorList([N, SMALL], **{p: [t[:n] for t, n in zip(x, (N, SMALL))] for p, x in back.items()}))
    for k, lo, hi in WINDOWS:
        x = window(host, lo, hi)
        want = {"master": x["master"]}
        for name in ("m", "v"):
            codes, scale = R.encode(R.blocks_of(x[name]), name, HALF)
            want[name] = R.decode(codes, scale, name).reshape(-1)[:hi - lo]
        for p in parts:
            parity.assert_bits_equal(back[p][k][lo:hi].cpu().numpy(), want[p], f"{p} {k} {lo}")
    for p in parts:
        for t, n in zip(back[p], (N, SMALL)):
            assert (t[n:] == 3.0).all(), p
