"""TensorList and ListDecision without a GPU: what they keep alive, what they wait for and what they refuse.  The list
entries are stand-ins with invented device addresses (nothing is launched); the table lies in host memory."""
import contextlib
import gc
import types
import weakref

import pytest
import torch

import mixed_precision_adam_amd as Z
from mixed_precision_adam_amd import driver as D

GPU = torch.device("cuda", 0)


class OnGpu:
    """As much of a GPU tensor as the host side looks at."""

    is_cuda = True
    next_address = 1 << 20

    def __init__(self, n, dtype=torch.float32, device=GPU):
        self.n, self.dtype, self.device = n, dtype, device
        self.at = OnGpu.next_address
        OnGpu.next_address += 4096 + 4 * n & ~0xFF

    def numel(self):
        return self.n

    def element_size(self):
        return self.dtype.itemsize

    def get_device(self):
        return self.device.index

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.at


class HostTorch:
    """torch, with a list's own device memory on the host and a log of what happens to it."""

    def __init__(self):
        self.log, self.capturing = [], False
        self.cuda = types.SimpleNamespace(synchronize=lambda device=None: self.log.append("wait for the device"),
                                          is_current_stream_capturing=lambda: self.capturing,
                                          current_device=lambda: 0, device=contextlib.nullcontext,
                                          current_stream=lambda: types.SimpleNamespace(synchronize=lambda: None))

    def __getattr__(self, name):
        return getattr(torch, name)

    def frombuffer(self, buffer, **kw):
        log = self.log

        class Staged(torch.Tensor):
            def to(self, device):
                assert device == GPU
                return Table.of(self, log)
        return torch.frombuffer(buffer, **kw).as_subclass(Staged)

    def zeros(self, n, dtype=torch.float32, device=None):
        return OnGpu(n, dtype, device)

    empty = zeros


class Table:
    """The device table."""

    @staticmethod
    def of(host, log):
        t = Table()
        t.bytes, t.log = bytearray(host.as_subclass(torch.Tensor).numpy().tobytes()), log
        t.keep = torch.empty(16, dtype=torch.uint8)
        return t

    def data_ptr(self):
        return self.keep.data_ptr()

    def __getitem__(self, part):
        table = self

        class Part:
            def copy_(self, host):
                table.log.append("table written")
                table.bytes[part] = host.as_subclass(torch.Tensor).numpy().tobytes()
        return Part()


@pytest.fixture
def host(monkeypatch):
    shim = HostTorch()
    monkeypatch.setattr(D, "torch", shim)
    return shim


@pytest.fixture
def queued(host, monkeypatch):
    """The calls that a step queues, by name, with what the decision was given: (max_norm, every group's settings)."""
    calls = []
    monkeypatch.setattr(D, "_current_raw_stream", lambda index: 0)
    monkeypatch.setattr(D, "zero_step_state_init", lambda *args: None)

    def decision(sq, flags, ranks, max_norm, hparams, state, groups, stream):
        calls.append(("decision", max_norm, [(h.lr, h.beta1, h.beta2, h.eps, h.weight_decay) for h in hparams]))
    monkeypatch.setattr(D, "zero_list_grad_sqnorm", lambda *args: calls.append(("norm",)))
    monkeypatch.setattr(D, "zero_list_decision_dev", decision)
    for name in ("zero_list_adamw_step_dev", "zero_list_adamw8_step_dev"):
        monkeypatch.setattr(D, name, lambda *args: calls.append(("update",)))
    return calls


def entries(sizes, dtype=torch.float32):
    return [OnGpu(n, dtype) for n in sizes]


def test_the_tensors_outlive_the_callers_lists(host):
    """Every address in the table belongs to a tensor that the list keeps, whatever becomes of the lists it was made
    from."""
    sizes = [8, 5000]
    for names in (("master", "m", "v"), ("state",), ("state8",)):
        made = {"grads": entries(sizes, torch.bfloat16), "params": entries(sizes, torch.bfloat16)}
        for k in names:
            made[k] = ([OnGpu(Z.zero_state8_bytes(n), torch.uint8) for n in sizes] if k == "state8" else
                       [OnGpu(Z.zero_state_tiled_numel(n)) for n in sizes] if k == "state" else entries(sizes))
        lst = D.TensorList(sizes, **made)
        refs = {k: [weakref.ref(t) for t in x] for k, x in made.items()}
        for x in made.values():
            x[0] = None
            x.clear()
        gc.collect()
        for k, x in refs.items():
            assert all(r() is not None for r in x), k
        del lst


def grads_of(table, n):
    """The gradient addresses that a table names."""
    return [int.from_bytes(table.bytes[64 * k:64 * k + 8], "little") for k in range(n)]


def test_new_gradients_wait_for_steps_in_flight(host):
    """A step queued on any stream, or a graph's replay, reads the table and the gradients that it names: the table is
    rewritten and the old gradients are let go only when the device is idle."""
    sizes = [8, 5000]
    lst = D.TensorList(sizes, entries(sizes), entries(sizes), master=entries(sizes), m=entries(sizes),
                       v=entries(sizes))
    old = [weakref.ref(g) for g in lst._grads]
    alive_at = []

    class Watched(list):
        def append(self, what):
            alive_at.append((what, all(r() is not None for r in old)))
    for target in (host, lst.table):
        target.log = Watched()
    new = entries(sizes, torch.bfloat16)
    lst.set_grads(new)
    assert alive_at == [("wait for the device", True), ("table written", True)]
    gc.collect()
    assert all(r() is None for r in old)
    assert grads_of(lst.table, 2) == [g.at for g in new]


def test_new_gradients_are_refused_while_capturing(host):
    sizes = [8, 5000]
    lst = D.TensorList(sizes, entries(sizes))
    before, named = list(lst._grads), bytes(lst.table.bytes)
    host.log.clear()
    host.capturing = True
    with pytest.raises(RuntimeError, match="captur"):
        lst.set_grads(entries(sizes))
    assert host.log == [] and lst._grads == before and bytes(lst.table.bytes) == named
    assert [r.grad for r in lst._recs] == [g.at for g in before]


def test_gradients_that_the_device_never_got_are_not_taken(host):
    """An error of the wait or of the copy leaves the list with the gradients that the device's table names."""
    sizes = [8, 5000]
    for failing in ("wait", "copy"):
        lst = D.TensorList(sizes, entries(sizes))
        before, staged = list(lst._grads), bytes(lst._host)

        def fails(*args):
            raise RuntimeError("device error")

        class Failing(list):
            append = fails
        if failing == "wait":
            host.cuda.synchronize = fails
        else:
            host.cuda.synchronize = lambda device=None: None
            lst.table.log = Failing()
        with pytest.raises(RuntimeError, match="device error"):
            lst.set_grads([None, OnGpu(5000)])
        assert lst._grads == before and bytes(lst._host) == staged, failing
        assert [r.grad for r in lst._recs] == [g.at for g in before]


def whole(sizes, n_groups=1):
    return D.TensorList(sizes, entries(sizes), entries(sizes), master=entries(sizes), m=entries(sizes),
                        v=entries(sizes), groups=[k % n_groups for k in range(len(sizes))], n_groups=n_groups)


def test_clipping_is_the_configurations(queued):
    """max_norm as DeviceDecision takes it, from the configuration; an argument of its own goes first."""
    def clipped(*cfgs, **kw):
        queued.clear()
        D.ListDecision(whole([8, 5000], len(cfgs)), list(cfgs), **kw).step()
        return queued[1][1]
    assert clipped(D.AdamWConfig()) == D.AdamWConfig().max_norm
    for norm in (0.0, 0.1, 2.0):
        assert clipped(D.AdamWConfig(max_norm=norm)) == norm
        assert clipped(D.AdamWConfig(max_norm=norm), D.AdamWConfig(lr=1.0, max_norm=norm)) == norm
        assert clipped(D.AdamWConfig(max_norm=0.3), max_norm=norm) == norm
    assert clipped(D.AdamWConfig(max_norm=0.1), D.AdamWConfig(max_norm=0.2), max_norm=0.5) == 0.5
    with pytest.raises(ValueError, match="max_norm"):
        clipped(D.AdamWConfig(max_norm=0.1), D.AdamWConfig(max_norm=0.2))


def test_a_changed_configuration_is_the_next_steps(queued):
    """A learning-rate schedule sets cfg.lr between steps, as with DeviceDecision, which reads its configuration at
    every step.  What a program sets in `hparams` or `max_norm` itself stays until the configuration changes."""
    cfgs = [D.AdamWConfig(lr=1e-3), D.AdamWConfig(lr=2e-3, weight_decay=0.0)]
    run = D.ListDecision(whole([8, 5000], 2), cfgs)

    def step():
        queued.clear()
        run.step()
        assert [c[0] for c in queued] == ["norm", "decision", "update"]
        return queued[1]

    def want(norm):
        return ("decision", norm, [(c.lr, c.beta1, c.beta2, c.eps, c.weight_decay) for c in cfgs])
    assert step() == want(1.0)
    cfgs[0].lr = 5e-4
    assert step() == want(1.0)
    cfgs[1].beta1, cfgs[1].beta2, cfgs[1].eps, cfgs[1].weight_decay = 0.8, 0.95, 1e-6, 0.2
    assert step() == want(1.0)
    for c in cfgs:
        c.max_norm = 0.25
    assert step() == want(0.25)
    run.hparams[0].lr, run.max_norm = 7e-4, 0.5
    _, norm, groups = step()
    assert norm == 0.5 and groups[0][0] == 7e-4
    cfgs[0].lr = 1e-4
    assert step() == want(0.5)
    cfgs[0].max_norm = 0.125
    queued.clear()
    with pytest.raises(ValueError, match="max_norm"):
        run.step()
    assert queued == []
    cfgs[1].max_norm = 0.125
    assert step() == want(0.125)


def test_a_given_max_norm_stays(queued):
    cfg = D.AdamWConfig(max_norm=0.1)
    run = D.ListDecision(whole([8]), [cfg], max_norm=0.5)
    cfg.max_norm, cfg.lr = 0.2, 3e-4
    run.step()
    assert queued[1][1] == 0.5 and queued[1][2][0][0] == 3e-4


def test_buffers_and_streams_of_another_gpu_are_refused(host, queued):
    """The kernels run on the list's GPU: an output, a step state or a stream of another one never reaches them."""
    there = torch.device("cuda", 1)
    lst = whole([8, 5000])
    sq, flag = OnGpu(1, torch.float64), OnGpu(1, torch.int32)
    state, groups = OnGpu(16, torch.float64), OnGpu(12)
    far = {x: OnGpu(x.n, x.dtype, there) for x in (sq, flag, state, groups)}
    stream = types.SimpleNamespace(cuda_stream=0, device=there)
    for call in (lambda: lst.grad_sqnorm(far[sq], flag), lambda: lst.grad_sqnorm(sq, far[flag]),
                 lambda: lst.adamw_dev(far[state], groups), lambda: lst.adamw_dev(state, far[groups]),
                 lambda: lst.grad_sqnorm(sq, flag, stream), lambda: lst.adamw_dev(state, groups, stream=stream),
                 lambda: lst.adamw(None, stream=stream), lambda: lst.pack8(lst, stream=stream),
                 lambda: lst.unpack8(lst, stream=stream),
                 lambda: D.ListDecision(lst, [D.AdamWConfig()]).step(stream)):
        with pytest.raises(ValueError, match="cuda:1"):
            call()
    assert queued == []
    near = types.SimpleNamespace(cuda_stream=0, device=GPU)
    lst.grad_sqnorm(sq, flag, near)
    lst.adamw_dev(state, groups, near)
    lst.grad_sqnorm(sq.at, flag.at, 0)
    assert len(queued) == 3


def test_steps_need_a_list_that_the_update_takes(queued):
    """Refused when made: at a step, the decision would have been queued (and counted) before the update's refusal."""
    sizes = [8, 5000]
    e = entries
    for lst in (D.TensorList(sizes, e(sizes)), D.TensorList(sizes, e(sizes), e(sizes)),
                D.TensorList(sizes, e(sizes), master=e(sizes), m=e(sizes), v=e(sizes)),
                D.TensorList(sizes, e(sizes), e(sizes), master=e(sizes), m=e(sizes)),
                D.TensorList(sizes, e(sizes), [OnGpu(8), None], master=e(sizes), m=e(sizes), v=e(sizes))):
        with pytest.raises(ValueError, match="param"):
            D.ListDecision(lst, [D.AdamWConfig()])
    for lst in (whole(sizes), D.TensorList([], []), D.TensorList(sizes, e(sizes), e(sizes), state8=[
            OnGpu(Z.zero_state8_bytes(n), torch.uint8) for n in sizes])):
        D.ListDecision(lst, [D.AdamWConfig()]).step()


def test_missing_buffers_and_other_libraries_streams(host, queued, monkeypatch):
    """A missing output is the library's refusal, and a stream may be any object with a handle."""
    lst = whole([8, 5000])
    lst.grad_sqnorm(OnGpu(1, torch.float64), OnGpu(1, torch.int32), types.SimpleNamespace(cuda_stream=0))
    assert queued == [("norm",)]
    monkeypatch.setattr(D, "zero_list_grad_sqnorm", Z.zero_list_grad_sqnorm)
    monkeypatch.setattr(D, "zero_list_adamw_step_dev", Z.zero_list_adamw_step_dev)
    for call in (lambda: lst.grad_sqnorm(None, OnGpu(1, torch.int32), 0),
                 lambda: lst.grad_sqnorm(OnGpu(1, torch.float64), None, 0),
                 lambda: lst.adamw_dev(None, OnGpu(12), 0), lambda: lst.adamw_dev(OnGpu(32), None, 0)):
        with pytest.raises(Z.ZeroError):
            call()
