"""The operators over lists on the GPU, against the plain forms of tests/list_reference.py.

Tolerances.  The update is a fixed sequence of fp32 operations, each correctly rounded, so master and moments, and the
8-bit codes and scales, are compared bit for bit; a 16-bit parameter is the rounding of that master.  The master of the
8-bit update has a tolerance of its own (assert_master8).  The norm's squares are exact in
fp64 and its sums are of non-negative terms, so any order is within n·2^-53 of the exact sum."""
import math

import numpy as np
import pytest
import torch

from tests import list_reference as R
from tests import parity

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mixed_precision_adam_amd as Z
    from mixed_precision_adam_amd.driver import (AdamWConfig, DeviceDecision, ListDecision, RankShard, TensorList)

DEV = "cuda:0"
FLOATS = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = [1, 3, 4, 5, 0, 255, 256, 257, 1023, 1024, 1025, 4095, 4096, 4097, 16385, 70001]
CFG = [dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1),
       dict(lr=3e-4, beta1=0.8, beta2=0.95, eps=1e-6, weight_decay=0.0)]
GUARD = 16  # sentinel elements on both sides of every buffer


class Guarded:
    """GPU tensors that start `shift` elements past a 16-byte boundary, between sentinels that must survive."""

    def __init__(self):
        self.held = []

    def __call__(self, host, shift=0):
        n = host.numel()
        item = host.element_size()
        lead = max(GUARD, 16 // item)
        buf = torch.full((lead + shift + n + GUARD,), 77, dtype=host.dtype, device=DEV)
        t = buf[lead + shift:lead + shift + n]
        t.copy_(host)
        self.held.append((buf, lead + shift, n))
        return t

    def check(self):
        for buf, lo, n in self.held:
            assert (buf[:lo] == 77).all() and (buf[lo + n:] == 77).all(), "a buffer's surroundings were written"


def hparams(step=1, grad_scale=1.0, groups=2):
    return Z.zero_list_hparams([dict(c, step=step, grad_scale=grad_scale) for c in CFG[:groups]])


def grads_host(n, dtype, rng, scale=1.0):
    g = torch.from_numpy(rng.standard_normal(n).astype(np.float32) * np.float32(1e-3 * scale))
    if n > 300:
        g[100:140] = 0.0
        g[7] *= 1e3
    return g.to(dtype)


def assert_bits_equal(got, want, what):
    """The same bits; a NaN equals a NaN (IEEE 754 leaves its sign and payload open, and host and GPU differ in
    them)."""
    got, want = np.asarray(got).reshape(-1), np.asarray(want).reshape(-1)
    if want.dtype == np.float32:
        nan = np.isnan(want)
        assert np.array_equal(np.isnan(got), nan), what
        got, want = got[~nan], want[~nan]
    parity.assert_bits_equal(got, want, what)


def param_bits(t):
    """The bits of parameters, every NaN as one pattern."""
    b = bits(t).copy()
    b[torch.isnan(t.detach().cpu()).numpy()] = -1
    return b


def assert_master8(got, want, p0, m, v, s, what):
    """The master of the 8-bit update against the fp32 form's, u = 2^-24.  The step step_size·m/d: the kernel's root,
    reciprocal of bc2_sqrt and reciprocal of d are within 2u each, the fused sum and two products u each: 9u; the
    plain form rounds five times: 5u; 14u together, 15 with the products of errors.  p·decay - step: the kernel rounds
    once, the plain form twice, each u of |p| or of the result."""
    got, want = got.astype(np.float64), want.astype(np.float64)
    step = s["step_size"] * np.abs(m.astype(np.float64)) / (np.sqrt(v.astype(np.float64)) / s["bc2_sqrt"] + s["eps"])
    far = np.abs(got - want) > 2.0**-24 * (15 * step + 3 * np.maximum(np.abs(p0), np.abs(want)))
    assert not far.any(), f"{what}: {far.sum()} of {far.size}, got {got[far][:3]} want {want[far][:3]}"


def bits(t):
    k = t.element_size()
    return t.detach().cpu().contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[k]).numpy()


# ---------------------------------------------------------------------- norm


@pytest.mark.parametrize("dtype", sorted(FLOATS))
@pytest.mark.parametrize("shift", [0, 1, 2, 3, 5])
@pytest.mark.parametrize("more", [[], [200_003], [11] * 60])  # one launch; too many elements for it; too many chunks
def test_norm(dtype, shift, more):
    rng = np.random.default_rng(shift)
    guard, sizes = Guarded(), SIZES + more
    host = [grads_host(n, FLOATS[dtype], rng) for n in sizes]
    grads = [guard(h, shift) for h in host]
    grads[7] = None  # no gradient in this step
    out = torch.zeros(2, dtype=torch.float64, device=DEV)
    lst = TensorList(sizes, grads)
    for _ in range(2):
        out.fill_(3.0)
        lst.grad_sqnorm(out[:1], out[1:].view(torch.int32))
        want = math.fsum(float(x) ** 2 for k, h in enumerate(host) if k != 7 for x in h.float())
        got, n = float(out[0]), sum(sizes)
        assert abs(got - want) <= n * 2.0**-53 * want
        assert int(out[1:].view(torch.int32)[0]) == 0
    guard.check()


@pytest.mark.parametrize("dtype", sorted(FLOATS))
@pytest.mark.parametrize("one_launch", [True, False])
def test_norm_flags_a_non_finite_gradient_anywhere(dtype, one_launch):
    sizes = [1, 5, 70001 if one_launch else 300_001]
    host = [torch.ones(n, dtype=FLOATS[dtype]) for n in sizes]
    out = torch.zeros(2, dtype=torch.float64, device=DEV)
    for value in (math.inf, -math.inf, math.nan):
        for k, i in ((0, 0), (1, 4), (2, 0), (2, 16384), (2, sizes[2] - 1)):
            host[k][i] = value
            TensorList(sizes, [h.to(DEV) for h in host]).grad_sqnorm(out[:1], out[1:].view(torch.int32))
            assert int(out[1:].view(torch.int32)[0]) == 1, (value, k, i)
            host[k][i] = 1.0
    largest = torch.finfo(FLOATS[dtype]).max  # finite gradients whose squares stay finite in fp64
    n = 4 if one_launch else 2**18
    TensorList([n], [torch.full((n,), largest, dtype=FLOATS[dtype], device=DEV)]).grad_sqnorm(
        out[:1], out[1:].view(torch.int32))
    want = n * float(largest) ** 2  # 48 significant bits: sums of more than 32 of them are rounded
    assert abs(float(out[0]) - want) <= n * 2.0**-53 * want and int(out[1:].view(torch.int32)[0]) == 0


def test_norm_of_nothing_is_zero():
    out = torch.full((2,), 3.0, dtype=torch.float64, device=DEV)
    for lst in (TensorList([]), TensorList([0, 0], [torch.zeros(0, device=DEV)] * 2), TensorList([5], [None])):
        out.fill_(3.0)
        lst.grad_sqnorm(out[:1], out[1:].view(torch.int32))
        assert float(out[0]) == 0.0 and int(out[1:].view(torch.int32)[0]) == 0


# ---------------------------------------------------------------------- AdamW, fp32 state


class List32:
    """A list with fp32 state on the GPU and its plain copy on the host."""

    def __init__(self, sizes, grad, param, layout, shift, seed, absent=(), groups=2):
        rng = np.random.default_rng(seed)
        self.sizes, self.guard, self.layout = sizes, Guarded(), layout
        self.group = [k % groups for k in range(len(sizes))]
        self.absent = set(absent)
        self.p = [(rng.standard_normal(n) * 0.02).astype(np.float32) for n in sizes]
        self.m = [(rng.standard_normal(n) * 3e-4).astype(np.float32) for n in sizes]
        self.v = [(rng.random(n) * 1e-6).astype(np.float32) for n in sizes]
        for m, v in zip(self.m, self.v):  # an embedding row that no token met
            m[100:120] = 0
            v[100:120] = 0
        self.grad_t, self.rng = FLOATS[grad], rng
        self.param = [self.guard(torch.from_numpy(p).to(FLOATS[param]), shift) for p in self.p]
        self.shift = shift
        if layout == "arrays":
            self.held = {k: [self.guard(torch.from_numpy(x), shift) for x in xs]
                         for k, xs in (("master", self.p), ("m", self.m), ("v", self.v))}
        else:
            self.held = {"state": [self.guard(torch.full((Z.zero_state_tiled_numel(n),), 5.0)) for n in sizes]}
            for n, st, p, m, v in zip(sizes, self.held["state"], self.p, self.m, self.v):
                Z.zero_state_tile(*[torch.from_numpy(x).to(DEV) for x in (p, m, v)], st, n)
        self.new_grads()
        self.list = TensorList(sizes, self.grads, self.param, groups=self.group, n_groups=groups, **self.held)

    def new_grads(self, scale=1.0):
        self.g = [grads_host(n, self.grad_t, self.rng, scale) for n in self.sizes]
        self.grads = [None if k in self.absent else self.guard(g, self.shift) for k, g in enumerate(self.g)]

    def plain_step(self, step, grad_scale):
        for k, g in enumerate(self.g):
            if k not in self.absent:
                s = R.scalars(**CFG[self.group[k]], grad_scale=grad_scale, step=step)
                self.p[k], self.m[k], self.v[k] = R.adamw(g.float().numpy(), self.p[k], self.m[k], self.v[k], s)

    def state(self, k):
        n = self.sizes[k]
        if self.layout == "arrays":
            return [self.held[x][k].cpu().numpy() for x in ("master", "m", "v")]
        out = [torch.empty(n, device=DEV) for _ in range(3)]
        Z.zero_state_untile(self.held["state"][k], *out, n)
        return [x.cpu().numpy() for x in out]

    def check(self, what=""):
        torch.cuda.synchronize()
        self.guard.check()
        for k, n in enumerate(self.sizes):
            for name, got, want in zip(("master", "m", "v"), self.state(k), (self.p[k], self.m[k], self.v[k])):
                assert_bits_equal(got, want, f"{what} tensor {k} ({n}) {name}")
            want = torch.from_numpy(self.p[k]).to(self.param[k].dtype)
            assert_bits_equal(param_bits(self.param[k]), param_bits(want), f"{what} tensor {k} ({n}) param")
            if self.layout == "tiled" and n:  # the padding keeps its bits
                tiles = self.held["state"][k].view(-1, 3, 1024)
                assert (tiles[-1, :, (n - 1) % 1024 + 1:] == 5.0).all()


@pytest.mark.parametrize("layout", ["arrays", "tiled"])
@pytest.mark.parametrize("grad", sorted(FLOATS))
@pytest.mark.parametrize("param", sorted(FLOATS))
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_adamw(layout, grad, param, shift):
    x = List32(SIZES, grad, param, layout, shift, seed=shift, absent=(6,))
    x.param[6].copy_(torch.from_numpy(x.p[6]))
    for step, gscale in ((1, 1.0), (2, 0.25), (1000, 2.0**-16)):
        if step > 1:
            x.new_grads(1 / gscale)
            x.list.set_grads(x.grads)
        x.list.adamw(hparams(step, gscale))
        x.plain_step(step, gscale)
        x.check(f"step {step}")


def test_adamw_is_the_flat_update():
    """One tensor in the list, the same bits as the flat tiled update."""
    n = 100_003
    x = List32([n], "bf16", "bf16", "tiled", 0, seed=9, groups=1)
    state, param = x.held["state"][0].clone(), torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    Z.zero_adamw_step_tiled(x.grads[0], Z.ZERO_BF16, state, param, n, **CFG[0], grad_scale=0.5, step=3)
    x.list.adamw(hparams(3, 0.5, groups=1))
    assert_bits_equal(bits(x.held["state"][0]), bits(state), "state")
    assert_bits_equal(bits(x.param[0]), bits(param), "param")


def test_adamw_over_many_tensors():
    """More tensors than any launch has workgroups per XCD group, one of them over several launches' worth of tiles
    of the others."""
    rng = np.random.default_rng(4)
    sizes = [int(n) for n in np.exp(rng.uniform(0, 9, 700))] + [1_500_001]
    x = List32(sizes, "bf16", "bf16", "arrays", 1, seed=4)
    x.list.adamw(hparams(2))
    x.plain_step(2, 1.0)
    x.check()


def test_adamw_mixed_list():
    """Every tensor with formats, layout, group and alignment of its own, in one list."""
    rng = np.random.default_rng(12)
    guard, tensors, parts = Guarded(), [], []
    kinds = [(g, p, lay) for g in FLOATS for p in FLOATS for lay in ("arrays", "tiled")]
    for k, (grad, param, layout) in enumerate(kinds):
        x = List32([700 + 301 * k], grad, param, layout, k % 4, seed=40 + k, groups=1)
        x.group = [int(rng.integers(0, 2))]
        held = {f: v[0] for f, v in x.held.items()}
        held["state"] = held.pop("master", held.get("state"))
        code = {torch.bfloat16: Z.ZERO_BF16, torch.float16: Z.ZERO_FP16, torch.float32: Z.ZERO_FP32}
        tensors.append(dict(numel=x.sizes[0], grad=x.grads[0], param=x.param[0], gdt=code[FLOATS[grad]],
                            pdt=code[FLOATS[param]], group=x.group[0],
                            layout=Z.ZERO_STATE_TILED if layout == "tiled" else Z.ZERO_STATE_ARRAYS, **held))
        parts.append(x)
    lst, table = Z.zero_list_plan(tensors, 2)
    table_dev = torch.frombuffer(table, dtype=torch.uint8).to(DEV)
    lst.table_dev = table_dev.data_ptr()
    Z.zero_list_adamw_step(lst, hparams(4))
    ws = torch.empty(Z.zero_list_grad_sqnorm_workspace_bytes(lst), dtype=torch.uint8, device=DEV)
    out = guard(torch.zeros(1, dtype=torch.float64))
    flag = guard(torch.zeros(1, dtype=torch.int32))
    Z.zero_list_grad_sqnorm(lst, ws, ws.numel(), out, flag)
    want = math.fsum(float(v) ** 2 for x in parts for v in x.g[0].float())
    assert abs(float(out[0]) - want) <= lst.numel * 2.0**-53 * want and int(flag[0]) == 0
    for k, x in enumerate(parts):
        x.plain_step(4, 1.0)
        x.check(f"{kinds[k]}")
    guard.check()


@pytest.mark.parametrize("param", ["bf16", "fp16"])
@pytest.mark.parametrize("eight", [False, True])
def test_parameter_rounding(param, eight):
    """Masters on and beside every rounding boundary of the format, zeros, subnormals, infinities and NaN, left as they
    are by a learning rate of zero: each parameter is the master's nearest value, ties to even."""
    if param == "fp16":
        p = parity.f16_probe_bits(20_000).view(np.float32)
    else:
        b = np.arange(1 << 16, dtype=np.uint32) << 16
        p = np.concatenate([b, b + 0x7FFF, b + 0x8000, b + 0x8001, b + 1]).view(np.float32)
    n = len(p)
    zero = np.zeros(n, np.float32)
    hp = Z.zero_list_hparams([dict(CFG[0], lr=0.0)])
    x = (List8 if eight else List32)([n], "bf16", param, **({} if eight else dict(layout="tiled", shift=0)), seed=0,
                                     groups=1)
    src = x.src if eight else x
    st = torch.from_numpy(p).to(DEV)
    if eight:
        TensorList([n], master=[st], m=[torch.from_numpy(zero).to(DEV)], v=[torch.from_numpy(zero).to(DEV)]).pack8(
            x.list)
    else:
        Z.zero_state_tile(st, *[torch.from_numpy(zero).to(DEV)] * 2, x.held["state"][0], n)
    x.list.adamw(hp)
    # (p·decay - step turns -0 into +0 where the step is -0, as the formula does: the master says which)
    master = x.host(0).master.copy() if eight else x.state(0)[0]
    assert np.array_equal(master, p, equal_nan=True)
    assert_bits_equal(param_bits(src.param[0]), param_bits(torch.from_numpy(master).to(FLOATS[param])), param)


@pytest.mark.parametrize("layout", ["arrays", "tiled"])
def test_adamw_extreme_values(layout):
    """Infinities, NaN, subnormals and the largest numbers do what the plain form does."""
    special = np.array([0.0, -0.0, np.inf, -np.inf, np.nan, 1e-45, -1e-40, 3.4e38, -3.4e38, 1e-20], np.float32)
    n = len(special) * 103
    x = List32([n], "fp32", "fp32", layout, 0, seed=3, groups=1)
    x.g[0] = torch.from_numpy(np.resize(special, n))
    x.grads[0].copy_(x.g[0])
    x.list.adamw(hparams(1, groups=1))
    x.plain_step(1, 1.0)
    for got, want in zip(x.state(0) + [x.param[0].cpu().numpy()], (x.p[0], x.m[0], x.v[0], x.p[0])):
        assert_bits_equal(got, want, "special values")


# ---------------------------------------------------------------------- 8-bit moments


class List8:
    """A list with 8-bit state packed from fp32 moments, and its plain form (tests.list_reference.State8)."""

    def __init__(self, sizes, grad="bf16", param="bf16", shift=0, seed=0, absent=(), groups=2, moments=None):
        self.src = List32(sizes, grad, param, "arrays", shift, seed, absent, groups)
        if moments is not None:
            for k, (m, v) in enumerate(moments):
                self.src.held["m"][k].copy_(torch.from_numpy(m))
                self.src.held["v"][k].copy_(torch.from_numpy(v))
                self.src.m[k], self.src.v[k] = m, v
        self.sizes, self.shift = sizes, shift
        self.state = [self.src.guard(torch.full((Z.zero_state8_bytes(n),), 9, dtype=torch.uint8)) for n in sizes]
        self.list = TensorList(sizes, self.src.grads, self.src.param, groups=self.src.group, n_groups=groups,
                               state8=self.state)
        self.src.list.pack8(self.list)

    def host(self, k):
        return R.State8(self.state[k].cpu().numpy(), self.sizes[k])

    def block0(self, k):
        return sum(-(-n // 4096) * 16 for n in self.sizes[:k])

    def check_padding(self):
        self.src.guard.check()
        for n, st in zip(self.sizes, self.state):
            if n % 4096:
                last = st.view(-1, 24704)[-1]
                cnt = n % 4096
                assert (last[4 * cnt:16384] == 9).all()
                for lo in (16384, 20480):
                    assert (last[lo + cnt:lo + 4096] == 9).all()
                used = -(-cnt // 256)
                for lo in (24576, 24640):
                    assert (last[lo + 4 * used:lo + 64] == 9).all()


def same_blocks(st, codes_m, codes_v, scale_m, scale_v, n, what):
    for name, got, want in (("m", st.m, codes_m), ("v", st.v, codes_v)):
        assert_bits_equal(got.reshape(-1)[:n], want.reshape(-1)[:n], f"{what} {name} codes")
    assert_bits_equal(st.scale_m, scale_m, f"{what} m scales")
    assert_bits_equal(st.scale_v, scale_v, f"{what} v scales")


@pytest.mark.parametrize("layout", ["arrays", "tiled"])
@pytest.mark.parametrize("shift", [0, 1])
def test_pack_and_unpack(layout, shift):
    src = List32(SIZES, "bf16", "bf16", layout, shift, seed=2)
    state = [src.guard(torch.full((Z.zero_state8_bytes(n),), 9, dtype=torch.uint8)) for n in SIZES]
    lst = TensorList(SIZES, state8=state)
    src.list.pack8(lst)
    back = {k: [src.guard(torch.full((n,), 3.0), shift) for n in SIZES] for k in ("master", "m", "v")}
    lst.unpack8(TensorList(SIZES, **back))
    src.check("the source is not touched")
    for k, n in enumerate(SIZES):
        st = R.State8(state[k].cpu().numpy(), n)
        half = 1 << 19
        cm, sm = R.encode(R.blocks_of(src.m[k]), "m", half) if n else (st.m, st.scale_m)
        cv, sv = R.encode(R.blocks_of(src.v[k]), "v", half) if n else (st.v, st.scale_v)
        same_blocks(st, cm, cv, sm, sv, n, f"tensor {k}")
        assert_bits_equal(st.master, src.p[k], "master")
        m, v = st.moments()
        for name, want in (("master", src.p[k]), ("m", m), ("v", v)):
            assert_bits_equal(back[name][k].cpu().numpy(), want, f"unpacked {name}")
        # against 64 bits: half a step, 2^-4 of the value (2^-10 of the top step among subnormals), plus the fp32
        # roundings of the scale, the position and the product
        for x, got, top, tiny in ((src.m[k], m, 448.0, 2.0**-10), (src.v[k], v, 1.875, 2.0**-34)):
            peak = np.repeat(np.abs(R.blocks_of(x)).max(axis=1), 256)[:n].astype(np.float64) if n else x
            bound = np.maximum(np.abs(x) * 2.0**-4, peak / top * tiny) * (1 + 1e-5) + peak * 2.0**-22
            if x is src.v[k]:
                bound = np.where(x > 0, np.maximum(bound, peak / top * 2.0**-33), bound)
            assert (np.abs(got - x.astype(np.float64)) <= bound).all()


@pytest.mark.parametrize("missing", ["master", "m", "v"])
@pytest.mark.parametrize("n", [5001, 1_300_003])  # within one tile per compute unit, and past it
def test_conversion_passes_over_missing_parts(missing, n):
    src = List32([n], "bf16", "bf16", "arrays", 0, seed=1, groups=1)
    state = torch.zeros(Z.zero_state8_bytes(n), dtype=torch.uint8, device=DEV)
    lst = TensorList([n], state8=[state])
    TensorList([n], **{k: x for k, x in src.held.items() if k != missing}).pack8(lst)
    st = R.State8(state.cpu().numpy(), n)
    for name, got in zip(("m", "v", "master"), (*st.moments(), st.master)):
        assert (got == 0).all() if name == missing else (got != 0).any()
    back = {k: [torch.full((n,), 3.0, device=DEV)] for k in ("master", "m", "v") if k != missing}
    lst.unpack8(TensorList([n], **back))
    for name, want in zip(("m", "v", "master"), (*st.moments(), st.master)):
        if name != missing:
            assert_bits_equal(back[name][0].cpu().numpy(), want, name)
    with pytest.raises(Z.ZeroError, match="not whole"):
        TensorList([n], src.grads, src.param, **{k: x for k, x in src.held.items() if k != missing}).adamw(
            hparams(groups=1))


@pytest.mark.parametrize("grad", sorted(FLOATS))
@pytest.mark.parametrize("param", sorted(FLOATS))
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_adamw8(grad, param, shift):
    x = List8(SIZES, grad, param, shift, seed=5, absent=(6,))
    for step, seed in ((1, 0), (2, 2**64 - 1), (70000, 12345)):
        if step > 1:
            x.src.new_grads()
            x.list.set_grads(x.src.grads)
        before = [x.host(k) for k in range(len(SIZES))]
        kept = bits(x.src.param[6]).copy()
        x.list.adamw(hparams(step, 0.5), seed=seed)
        x.check_padding()
        assert (x.state[6].cpu().numpy() == before[6].raw).all() and (bits(x.src.param[6]) == kept).all()
        for k, n in enumerate(SIZES):
            if n == 0 or k == 6:
                continue
            s = R.scalars(**CFG[x.src.group[k]], grad_scale=0.5, step=step)
            g = x.src.g[k].float().numpy()
            p, cm, cv, sm, sv = R.adamw8(g, before[k], s, seed, step, x.block0(k))
            st = x.host(k)
            same_blocks(st, cm, cv, sm, sv, n, f"step {step} tensor {k}")
            _, m, v = R.adamw(g, before[k].master, *before[k].moments(), s)
            assert_master8(st.master, p, before[k].master, m, v, s, f"step {step} tensor {k} master")
            want = torch.from_numpy(st.master.copy()).to(x.src.param[k].dtype)
            assert_bits_equal(bits(x.src.param[k]), bits(want), f"tensor {k} param")


def test_adamw8_against_64_bits():
    """Every decoded moment lies within one step of the 64-bit value: a whole step is at most 2^-3 of the value."""
    n = 70001
    x = List8([n], "fp32", "fp32", seed=6, groups=1)
    st = x.host(0)
    m0, v0 = (a.astype(np.float64) for a in st.moments())
    s = R.scalars(**CFG[0], grad_scale=1.0, step=5)
    p, m, v = R.adamw(x.src.g[0].double().numpy(), st.master.astype(np.float64), m0, v0, s, np.float64)
    x.list.adamw(hparams(5, groups=1), seed=1)
    st = x.host(0)
    for got, want, top, tiny in zip(st.moments(), (m, v), (448.0, 1.875), (2.0**-9, 2.0**-33)):
        peak = np.repeat(np.abs(R.blocks_of(want)).max(axis=1), 256)[:n]
        bound = np.maximum(np.abs(want) * 2.0**-3, peak / top * tiny) * (1 + 1e-5) + peak * 2.0**-21
        assert (np.abs(got - want) <= bound).all()
    # The master, with u = 2^-24: p·decay - step takes the roundings of decay, the product and the difference (4u of
    # |p| with their second-order terms).  The step is step_size·m/d: m is a sum of two products that may cancel, so
    # its errors (each product and its scalar, the sum: 4u) count on the size of its terms, and gscale·g's (2u) with
    # them; v adds 6u, half of it after the root, and root, division, eps, m/d, step_size and their scalars 8: under
    # 30u of step_size·(b1·|m| + (1-b1)·|g|)/(d - eps) in all.
    g = np.abs(x.src.g[0].double().numpy())
    step = s["step_size"] * (s["b1"] * np.abs(m0) + s["omb1"] * g) / np.maximum(np.sqrt(v) / s["bc2_sqrt"], s["eps"])
    assert (np.abs(st.master - p) <= 2.0**-24 * (4 * np.abs(x.src.p[0]) + 30 * step)).all()


def test_adamw8_second_moment_follows_its_average():
    """With gradients of zero v decays by beta2 a step.  Rounding to nearest would leave it where it is (0.1% a step
    against codes 6 to 12% apart); rounded stochastically its mean over 65,536 elements follows.  Each step adds an
    error of mean zero and at most half a step's deviation (2^-4 relative) to an element: over 300 steps at most
    300^.5 · 2^-4 = 1.1 of its value, over 65,536 of them 0.42%; five times that allowed."""
    n, steps = 65536, 300
    v0 = np.full(n, 1e-6, np.float32)
    v0[::256] = 2e-6  # the peak of every block decays too
    x = List8([n], moments=[(np.zeros(n, np.float32), v0)], groups=1)
    start = x.host(0).moments()[1].astype(np.float64)
    x.src.grads[0].zero_()
    for t in range(1, steps + 1):
        x.list.adamw(hparams(t, groups=1), seed=77)
    ratio = x.host(0).moments()[1].astype(np.float64).mean() / start.mean()
    assert abs(ratio / 0.999**steps - 1) < 5 * 0.0042
    assert (x.host(0).moments()[1] > 0).all()


def test_adamw8_special_blocks():
    """A block of zeros, one whose peak is below 2^-110, a v that would round to zero, one outlier among tiny values,
    and non-finite moments: the plain form's codes and scales; a NaN or infinity shows in the whole block."""
    n = 8 * 256
    rng = np.random.default_rng(0)
    m = (rng.standard_normal(n) * 1e-4).astype(np.float32)
    v = (rng.random(n) * 1e-8).astype(np.float32)
    b = [slice(256 * k, 256 * (k + 1)) for k in range(8)]
    m[b[0]] = v[b[0]] = 0
    m[b[1]], v[b[1]] = 1e-34, 1e-36
    v[b[2]] = 1e-20
    v[512] = 1.0
    m[b[3]] = 1e-30
    m[800] = -1e30
    m[b[4]] = 3e38
    v[b[4]] = 3e38
    m[1300], v[1301] = np.nan, np.inf
    m[1600] = -np.inf
    v[1601] = np.nan
    x = List8([n], "fp32", "fp32", moments=[(m, v)], groups=1)
    half = 1 << 19
    with np.errstate(all="ignore"):
        cm, sm = R.encode(R.blocks_of(m), "m", half)
        cv, sv = R.encode(R.blocks_of(v), "v", half)
    st = x.host(0)
    for got, want in ((st.scale_m, sm), (st.scale_v, sv)):
        assert np.array_equal(got, want, equal_nan=True)
    for k in range(8):
        if k not in (5, 6):
            assert (st.m[k] == cm[k]).all() and (st.v[k] == cv[k]).all(), k
    gm, gv = st.moments()
    assert (gm[b[0]] == 0).all() and (gv[b[0]] == 0).all() and (gm[b[1]] == 0).all() and (gv[b[1]] == 0).all()
    assert (gv[b[2]] > 0).all()
    assert not np.isfinite(gm[b[5]]).any() and not np.isfinite(gv[b[5]]).any()
    assert not np.isfinite(gm[b[6]]).any() and not np.isfinite(gv[b[6]]).any()
    assert np.isfinite(gm[b[7]]).all() and np.isfinite(gv[b[7]]).all()
    # a step from there: finite blocks agree with the plain form
    x.src.grads[0].fill_(1e-5)
    x.list.adamw(hparams(3, groups=1), seed=4)
    s = R.scalars(**CFG[0], grad_scale=1.0, step=3)
    p, cm, cv, sm, sv = R.adamw8(np.full(n, 1e-5, np.float32), st, s, 4, 3, 0)
    new = x.host(0)
    for k in (0, 1, 2, 3, 4, 7):
        assert (new.m[k] == cm[k]).all() and (new.v[k] == cv[k]).all(), k
        assert new.scale_m[k] == sm[k] and new.scale_v[k] == sv[k]
        at = b[k]
        _, m1, v1 = R.adamw(np.full(256, 1e-5, np.float32), st.master[at], gm[at], gv[at], s)
        assert_master8(new.master[at], p[at], st.master[at], m1, v1, s, f"block {k} master")


def test_adamw8_least_eps():
    """An eps of zero in the device form counts as 1e-16: where both moments are held as zeros nothing moves."""
    n = 5000
    x = List8([n], "fp32", "fp32", moments=[(np.zeros(n, np.float32), np.zeros(n, np.float32))], groups=1)
    x.src.grads[0].zero_()
    run = ListDecision(x.list, [AdamWConfig(eps=0.0, weight_decay=0.0)], max_norm=0.0)
    run.step()
    assert run.read()["skip"] == 0
    assert_bits_equal(x.host(0).master, x.src.p[0], "master")


def test_adamw8_rounding_depends_on_its_arguments_alone():
    def run(seed, step):
        x = List8([70001], seed=8, groups=1)
        x.list.adamw(hparams(step, groups=1), seed=seed)
        return x.state[0].cpu().numpy()
    a = run(1, 2)
    assert (run(1, 2) == a).all()
    assert (run(2, 2) != a).any()


# ---------------------------------------------------------------------- together: norm, decision, update


def test_decision_scalars_of_every_group():
    """The decision of zero_step_decision_dev, and for each group the scalars it gives with that group's settings."""
    cfgs = [dict(lr=1e-3 * (k + 1), beta1=0.9 - 0.01 * k, beta2=0.999 - 0.001 * k, eps=1e-8 * (k + 1),
                 weight_decay=0.01 * k) for k in range(64)]
    hp = Z.zero_list_hparams(cfgs)
    sq = torch.tensor([9.0, 7.0], dtype=torch.float64, device=DEV)
    flags = torch.zeros(2, dtype=torch.int32, device=DEV)
    state, one = (torch.zeros(16, dtype=torch.float64, device=DEV) for _ in range(2))
    groups = torch.full((64 * 12,), 7.0, device=DEV)
    Z.zero_step_state_init(state, 4.0, 2)
    for step in range(3):
        Z.zero_list_decision_dev(sq, flags, 2, 0.5, hp, state, groups)
        for k in (0, 1, 63):
            Z.zero_step_state_init(one, 4.0, 2)
            for _ in range(step + 1):
                Z.zero_step_decision_dev(sq, flags, 2, 0.5, one, **cfgs[k])
            want, got = Z.read_step_state(one), Z.read_step_state(state)
            assert want["scalars"] == groups.view(64, 12)[k, :9].tolist()
            assert all(got[f] == want[f] for f in got if f != "scalars")
            if k == 0:
                assert got["scalars"] == want["scalars"]
    before = groups.clone()
    flags[1] = 1
    Z.zero_list_decision_dev(sq, flags, 2, 0.5, hp, state, groups)
    assert Z.read_step_state(state)["skip"] == 1 and torch.equal(groups, before)


@pytest.mark.parametrize("eight", [False, True])
def test_whole_steps(eight):
    """Norm, decision and update queued together, against the same steps taken from the host; an overflow skips
    everything, then the loss scale is halved."""
    kw = dict(seed=11, absent=(5,))
    x = List8(SIZES, "fp16", **kw) if eight else List32(SIZES, "fp16", "bf16", "tiled", 1, **kw)
    y = List8(SIZES, "fp16", **kw) if eight else List32(SIZES, "fp16", "bf16", "tiled", 1, **kw)
    lists = [(z.src if eight else z) for z in (x, y)]
    run = ListDecision(x.list, [AdamWConfig(**c) for c in CFG], max_norm=0.05, loss_scale=1024.0, seed=3)
    scale, t = 1024.0, 0
    for it in range(4):
        for z, src in zip((x, y), lists):
            src.rng = np.random.default_rng(100 + it)
            src.new_grads(scale)
            if it == 1:
                src.grads[15][69999] = math.inf
            z.list.set_grads(src.grads)
        before = [bits(s).copy() for s in (x.state if eight else x.held["state"])]
        run.step()
        got = run.read()
        total = math.fsum(float(v) ** 2 for k, g in enumerate(lists[0].g) if k != 5 for v in g.float())
        if it == 1:
            scale /= 2
            assert got["skip"] == 1 and got["loss_scale"] == scale and got["adam_step"] == t
            for s, b in zip(x.state if eight else x.held["state"], before):
                assert (bits(s) == b).all()
            continue
        t += 1
        assert got["skip"] == 0 and got["adam_step"] == t
        assert got["global_norm"] == pytest.approx(math.sqrt(total) / scale, rel=1e-10)
        y.list.adamw(hparams(t, got["grad_scale"]), seed=3)
        for a, b in zip(x.state if eight else x.held["state"], y.state if eight else y.held["state"]):
            assert_bits_equal(bits(a), bits(b), f"state, step {it}")
        for a, b in zip(lists[0].param, lists[1].param):
            assert_bits_equal(bits(a), bits(b), f"param, step {it}")


def test_whole_step_over_a_ranks_pieces():
    """A list of the pieces of rank 1's shard, stepped where they lie, gives the flattened step's state and
    parameters (no clipping: the two norms are summed in different orders)."""
    numels, world, rank = [5000, 17, 40_003, 64, 9001], 3, 1
    rng = np.random.default_rng(0)
    srcs = [grads_host(n, torch.bfloat16, rng).to(DEV) for n in numels]
    shard = RankShard(numels, world, rank, Z.ZERO_BF16, DEV, sources=srcs, tiled=True, fused=True)
    master = torch.from_numpy((rng.standard_normal(shard.n) * 0.02).astype(np.float32)).to(DEV)
    shard.load_master(master)
    cfg = AdamWConfig(max_norm=0.0)
    flat = DeviceDecision([shard], cfg)
    pieces = [(s.tensor, s.src_offset, s.dst_offset, s.numel) for s in shard.segments]
    p, m, v = master.clone(), torch.zeros_like(master), torch.zeros_like(master)
    param = torch.zeros(shard.n, dtype=torch.bfloat16, device=DEV)
    lst = TensorList([n for *_, n in pieces], [srcs[t][o:o + n] for t, o, _, n in pieces],
                     [param[d:d + n] for _, _, d, n in pieces],
                     **{k: [x[d:d + n] for _, _, d, n in pieces] for k, x in (("master", p), ("m", m), ("v", v))})
    run = ListDecision(lst, [cfg], max_norm=0.0)
    for _ in range(3):
        flat.step()
        run.step()
    for got, want in zip((p, m, v), shard.read_state()):
        assert_bits_equal(bits(got), bits(want), "state")
    assert_bits_equal(bits(param), bits(shard.param), "param")
    assert run.read()["global_norm"] == pytest.approx(flat.read()["global_norm"], rel=1e-12)


@pytest.mark.parametrize("eight", [False, True])
def test_captured_steps(eight):
    """A captured step replayed between eager work, every replay equal to an eager step of a second list."""
    sizes = [1, 5000, 70001]
    x = List8(sizes, seed=1) if eight else List32(sizes, "bf16", "bf16", "arrays", 0, seed=1)
    y = List8(sizes, seed=1) if eight else List32(sizes, "bf16", "bf16", "arrays", 0, seed=1)
    srcs = [(z.src if eight else z) for z in (x, y)]
    cfgs = [AdamWConfig(**c) for c in CFG]
    a, b = (ListDecision(z.list, cfgs, max_norm=0.05, seed=9) for z in (x, y))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        a.step(torch.cuda.current_stream())
    for it in range(5):
        if it == 3:  # the replays read what the table names by then
            for z, src in zip((x, y), srcs):
                src.grads = [torch.zeros_like(g) for g in src.grads]
                z.list.set_grads(src.grads)
        for src in srcs:
            for k, g in enumerate(src.grads):
                g.copy_(grads_host(sizes[k], g.dtype, np.random.default_rng(10 * it + k)))
        graph.replay()
        b.step()
        torch.randn(1000, device=DEV).sum()
        torch.cuda.synchronize()
        assert a.read()["adam_step"] == it + 1
        for k in range(3):
            got, want = ((x.state[k], y.state[k]) if eight else (x.held["master"][k], y.held["master"][k]))
            assert_bits_equal(bits(got), bits(want), f"replay {it} tensor {k}")
            assert_bits_equal(bits(srcs[0].param[k]), bits(srcs[1].param[k]), f"replay {it} param {k}")


def test_two_lists_on_two_streams():
    """Lists with buffers of their own run at the same time."""
    x, y = List32([500_003], "bf16", "bf16", "tiled", 0, seed=1, groups=1), List8([500_003], seed=2, groups=1)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    st = y.host(0)
    x.list.adamw(hparams(1, groups=1), stream=streams[0])
    y.list.adamw(hparams(1, groups=1), stream=streams[1], seed=6)
    torch.cuda.synchronize()
    x.plain_step(1, 1.0)
    x.check()
    s = R.scalars(**CFG[0], grad_scale=1.0, step=1)
    p, cm, cv, sm, sv = R.adamw8(y.src.g[0].float().numpy(), st, s, 6, 1, 0)
    same_blocks(y.host(0), cm, cv, sm, sv, 500_003, "second stream")


def test_first_step_on_another_stream():
    """A ListDecision made behind queued work steps at once on another stream as on its own."""
    big = torch.zeros(1 << 28, device=DEV)
    x, y = (List32([70_001], "bf16", "bf16", "tiled", 0, seed=4, groups=1) for _ in range(2))
    cfg = [AdamWConfig(**CFG[0])]
    plain = ListDecision(x.list, cfg, loss_scale=2.0)
    plain.step()
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(100):
        big.add_(1.0)
    run = ListDecision(y.list, cfg, loss_scale=2.0)
    run.step(stream=other)
    torch.cuda.synchronize()
    assert run.read() == plain.read()
    for a, b in zip(x.held["state"], y.held["state"]):
        assert_bits_equal(bits(a), bits(b), "state")


def test_state_read_after_a_step_on_another_stream():
    """What read() gives is the queued step's, whose stream is not the current one and busy."""
    big = torch.zeros(1 << 28, device=DEV)
    x = List32([70_001], "bf16", "bf16", "tiled", 0, seed=4, groups=1)
    run = ListDecision(x.list, [AdamWConfig(**CFG[0])], loss_scale=2.0)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        for _ in range(100):
            big.add_(1.0)
        run.step()
    assert run.read()["adam_step"] == 1


def test_tensor_list_refusals():
    g = torch.zeros(8, dtype=torch.bfloat16, device=DEV)
    f = torch.zeros(8, device=DEV)
    with pytest.raises(ValueError, match="entries"):
        TensorList([8, 8], [g])
    with pytest.raises(ValueError, match="GPU"):
        TensorList([8], [g.cpu()])
    with pytest.raises(ValueError, match="dtype"):
        TensorList([8], [g.double()])
    with pytest.raises(ValueError, match="dtype"):
        TensorList([8], [g], master=[g])
    with pytest.raises(ValueError, match="one kind"):
        TensorList([8], [g], master=[f], state8=[torch.zeros(Z.zero_state8_bytes(8), dtype=torch.uint8, device=DEV)])
    with pytest.raises(ValueError, match="contiguous"):
        TensorList([4], [g[::2]])
    with pytest.raises(ValueError, match="bytes"):
        TensorList([9], [g])
    with pytest.raises(ValueError, match="bytes"):
        TensorList([8], [g], state=[f])
    lst = TensorList([8], [g], [g.clone()], master=[f], m=[f.clone()], v=[f.clone()])
    with pytest.raises(ValueError, match="groups"):
        lst.adamw(hparams(groups=2))
    with pytest.raises(Z.ZeroError):
        lst.set_grads([f])  # the master itself
    assert lst._grads[0] is g and lst._recs[0].grad == g.data_ptr()  # what the table still names is kept
    with pytest.raises(ValueError, match="gradients"):
        lst.set_grads([g, g])


def test_a_models_parameters_step_as_torchs_optimizer():
    """A model's own parameters and gradients (new tensors at every backward), weights decayed and biases not, clipped:
    torch's AdamW and clip_grad_norm_ on a copy.  Both round every operation to fp32 in slightly different orders: a
    parameter's update of about lr differs by some ten units of 2^-24 a step, its own rounding by two."""
    torch.manual_seed(0)
    make = lambda: torch.nn.Sequential(torch.nn.Linear(37, 129), torch.nn.GELU(), torch.nn.Linear(129, 5)).to(DEV)  # noqa: E731
    model, copy = make(), make()
    copy.load_state_dict(model.state_dict())
    params, lr = list(model.parameters()), 1e-2
    state = {k: [torch.zeros_like(p) for p in params] for k in ("master", "m", "v")}
    for w, p in zip(state["master"], params):
        w.copy_(p.detach())
    opt = torch.optim.AdamW([dict(params=[p for p in copy.parameters() if p.dim() > 1], weight_decay=0.1),
                             dict(params=[p for p in copy.parameters() if p.dim() == 1], weight_decay=0.0)], lr=lr)
    tensors, steps = None, 4
    for t in range(steps):
        x = torch.randn(64, 37, device=DEV, generator=torch.Generator(DEV).manual_seed(t))
        for net in (model, copy):
            net.zero_grad(set_to_none=True)
            net(x).square().mean().backward()
        if tensors is None:
            tensors = TensorList([p.numel() for p in params], [p.grad for p in params], params, **state,
                                 groups=[0 if p.dim() > 1 else 1 for p in params], n_groups=2)
            run = ListDecision(tensors, [AdamWConfig(lr=lr, weight_decay=0.1), AdamWConfig(lr=lr, weight_decay=0.0)],
                               max_norm=0.1)
        else:
            tensors.set_grads([p.grad for p in params])
        run.step()
        norm = torch.nn.utils.clip_grad_norm_(copy.parameters(), 0.1)
        opt.step()
        # the two models' gradients differ by what their parameters do: the norms agree to 1e-4
        assert run.read()["global_norm"] == pytest.approx(float(norm), rel=1e-4)
        if t == 0:  # the same gradients on both sides
            for p, q, w in zip(params, copy.parameters(), state["master"]):
                assert torch.equal(p.detach(), w)
                assert (p - q).abs().max() <= 2.0**-24 * (4 * q.abs().max() + 40 * lr)
