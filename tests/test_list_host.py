"""Lists of tensors without a GPU: sizes, the plan's table, every refusal (checked on the host before anything is
launched), and the plain forms that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import mixed_precision_adam_amd as Z
from tests import list_reference as R

HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)


def tensor(at=0x100000, n=5000, **kw):
    """A well-formed entry with separate arrays, at invented addresses (the host checks never read them)."""
    step = 4 * n + 4096 & ~0xFFF
    t = dict(grad=at, param=at + step, state=at + 2 * step, m=at + 3 * step, v=at + 4 * step, numel=n,
             layout=Z.ZERO_STATE_ARRAYS)
    t.update(kw)
    return t


def refused(tensors, n_groups=1, word=""):
    with pytest.raises(Z.ZeroError) as e:
        Z.zero_list_plan(tensors, n_groups)
    assert e.value.status == Z.ZERO_ERR_INVALID and word in str(e.value), str(e.value)


def planned(tensors, n_groups=1):
    lst, table = Z.zero_list_plan(tensors, n_groups)
    lst.table_dev = 0x7000000
    return lst, table


def test_state8_bytes():
    per = 6 * 4096 + 2 * 4 * 16
    assert [Z.zero_state8_bytes(n) for n in (-1, 0, 1, 4096, 4097, 2**58 - 1, 2**58)] == \
        [0, 0, per, per, 2 * per, 2**46 * per, 0]


def test_structures_match_the_header(tmp_path):
    import os

    from tests.test_struct_layouts import ROOT, c_layout, check

    structs = {"zero_list_tensor": Z.zero_list_tensor, "zero_list": Z.zero_list,
               "zero_group_scalars": Z.zero_group_scalars}
    check(c_layout(tmp_path, os.path.join(ROOT, "include"), "zero_shard.h", structs), structs)


def test_table_covers_every_element_once():
    sizes = [1, 0, 1024, 5000, 16385, 70001]
    at, tensors = 0x100000, []
    for k, n in enumerate(sizes):
        tensors.append(tensor(at, n, group=k % 2))
        at += 0x1000000
    for layout, per in ((Z.ZERO_STATE_ARRAYS, None), (Z.ZERO_STATE_8BIT, None), (Z.ZERO_STATE_NONE, None)):
        for t in tensors:
            t["layout"] = layout
            if layout != Z.ZERO_STATE_ARRAYS:
                t["m"] = t["v"] = None
            if layout == Z.ZERO_STATE_NONE:
                t["state"] = None
        lst, table = Z.zero_list_plan(tensors, 2)
        assert lst.numel == sum(sizes) and lst.n_tensors == len(sizes) and lst.table_bytes == len(table)
        assert lst.grads_bytes == 64 * len(sizes)
        for off, count in ((lst.norm_offset, lst.norm_blocks), (lst.update_offset, lst.update_blocks)):
            rec = np.frombuffer(table, np.uint32, 2 * count, off).reshape(-1, 2)
            if layout == Z.ZERO_STATE_NONE and off == lst.update_offset and count == 0:
                continue
            for k, n in enumerate(sizes):  # chunks 0 .. c-1 of every tensor, in order
                chunks = rec[rec[:, 0] == k, 1]
                assert (chunks == np.arange(len(chunks))).all()
                assert (len(chunks) == 0) == (n == 0)
            assert (np.diff(rec[:, 0].astype(np.int64)) >= 0).all()


def test_lists_that_are_refused():
    refused([tensor(gdt=3)], word="gradient dtype")
    refused([tensor(pdt=-1)], word="parameter dtype")
    refused([tensor(layout=4)], word="layout")
    refused([tensor(numel=-1)], word="out of range")
    refused([tensor(numel=2**40 + 1)], word="out of range")
    refused([tensor(group=1)], word="group")
    refused([tensor(group=-1)], word="group")
    refused([tensor()], n_groups=0, word="n_groups")
    refused([tensor()], n_groups=Z.ZERO_LIST_MAX_GROUPS + 1, word="n_groups")
    refused([tensor(grad=0x100001)], word="aligned")
    refused([tensor(grad=0x100002, gdt=Z.ZERO_FP32)], word="aligned")
    refused([tensor(param=0x200001)], word="aligned")
    refused([tensor(m=0x300002)], word="misaligned state")
    refused([tensor(layout=Z.ZERO_STATE_TILED)], word="separate arrays")
    refused([tensor(layout=Z.ZERO_STATE_TILED, m=None, v=None, state=0x300008)], word="misaligned state")
    refused([tensor(layout=Z.ZERO_STATE_8BIT, m=None, v=None, state=0x300004)], word="misaligned state")
    refused([tensor(layout=Z.ZERO_STATE_TILED, m=None, v=None, state=None)], word="NULL state")
    refused([tensor(layout=Z.ZERO_STATE_NONE, m=None, v=None)], word="without a layout")
    refused([tensor(), tensor(0x900000, layout=Z.ZERO_STATE_8BIT, m=None, v=None)], word="one kind of state")
    refused([tensor(2**64 - 8192 & ~0xFFF, n=5000)], word="address space")


def test_overlaps_are_refused():
    a = tensor()
    refused([a, dict(a)], word="overlaps")                                       # the same tensor twice
    b = tensor(0x900000)
    refused([a, dict(b, param=a["param"] + 2 * 4999)], word="overlaps")          # the last parameter of a
    refused([a, dict(b, m=a["v"])], word="overlaps")
    refused([a, dict(b, grad=a["param"])], word="overlaps")                      # b's gradients are a's parameters
    refused([dict(a, param=a["grad"])], word="overlaps")
    refused([dict(a, pdt=Z.ZERO_FP32, param=a["state"])], word="overlaps")       # fp32 parameters as their own master
    t = tensor(layout=Z.ZERO_STATE_TILED, m=None, v=None)
    refused([dict(t, param=t["state"] + 4 * Z.zero_state_tiled_numel(5000) - 2)], word="overlaps")  # tile padding
    planned([a, dict(b, grad=a["grad"])])                                        # gradients may share memory
    planned([a, dict(b, param=a["param"] + 2 * 5000)])                           # touching is not overlapping
    planned([a, dict(a, numel=0)])                                               # nothing is read or written


def test_a_small_table_is_refused():
    recs = (Z.zero_list_tensor * 1)()
    recs[0].numel = 5000
    out, table = Z.zero_list(), (ctypes.c_char * 64)()
    need = Z.zero_list_table_bytes([dict(numel=5000)])
    assert need == 64 + 8 * 1  # a descriptor and one workgroup of the norm
    lib = Z.library()
    assert lib.zero_list_plan(ctypes.cast(recs, Z._P), 1, 1, table, need - 1, ctypes.byref(out)) == Z.ZERO_ERR_CAPACITY
    assert lib.zero_list_plan(ctypes.cast(recs, Z._P), 1, 1, None, need, ctypes.byref(out)) == Z.ZERO_ERR_INVALID
    assert lib.zero_list_plan(None, 1, 1, table, need, ctypes.byref(out)) == Z.ZERO_ERR_INVALID
    assert lib.zero_list_plan(ctypes.cast(recs, Z._P), -1, 1, table, need, ctypes.byref(out)) == Z.ZERO_ERR_INVALID


def test_repoint():
    a, b = tensor(), tensor(0x900000, 70001)
    lst, table = planned([a, b])
    before = bytes(table)
    Z.zero_list_repoint([dict(a, grad=None), dict(b, grad=0x5000000)], table, lst)
    assert table[lst.grads_bytes:] == before[lst.grads_bytes:] and table != before
    Z.zero_list_repoint([a, b], table, lst)
    assert bytes(table) == before
    for bad in ([a], [a, dict(b, numel=70000)], [b, a], [a, dict(b, param=a["param"])], [a, dict(b, param=None)],
                [dict(x, layout=Z.ZERO_STATE_8BIT, m=None, v=None) for x in (a, b)]):
        with pytest.raises(Z.ZeroError):
            Z.zero_list_repoint(bad, table, lst)
        assert bytes(table) == before  # nothing is written
    with pytest.raises(Z.ZeroError):
        Z.zero_list_repoint([a, b], bytearray(lst.grads_bytes - 1), lst)


def test_device_calls_refuse_before_they_launch():
    a = tensor()
    lst, _ = planned([a], 2)
    eight, _ = planned([tensor(layout=Z.ZERO_STATE_8BIT, m=None, v=None)], 2)
    hp = Z.zero_list_hparams([HP, HP])
    lib, inv = Z.library(), Z.ZERO_ERR_INVALID
    ref = ctypes.byref

    def word(rc, text):
        assert rc == inv and text in Z.zero_last_error(), Z.zero_last_error()

    word(lib.zero_list_adamw_step(None, hp, None), "list NULL")
    word(lib.zero_list_adamw_step(ref(Z.zero_list()), hp, None), "not planned")
    changed = Z.zero_list.from_buffer_copy(lst)
    changed.update_blocks += 1
    word(lib.zero_list_adamw_step(ref(changed), hp, None), "not planned")
    changed = Z.zero_list.from_buffer_copy(lst)
    changed.table_dev = None
    word(lib.zero_list_adamw_step(ref(changed), hp, None), "device table")
    changed.table_dev = 8
    word(lib.zero_list_adamw_step(ref(changed), hp, None), "device table")
    word(lib.zero_list_adamw_step(ref(lst), None, None), "hparams NULL")
    word(lib.zero_list_adamw_step(ref(eight), hp, None), "8-bit state")
    word(lib.zero_list_adamw8_step(ref(lst), hp, 0, None), "fp32 state")
    word(lib.zero_list_adamw_step(ref(planned([dict(a, param=None)])[0]), hp, None), "no param")
    word(lib.zero_list_adamw_step(ref(planned([dict(a, v=None)])[0]), hp, None), "not whole")
    for field, value in (("step", 0), ("beta1", 1.0), ("beta2", -0.1), ("lr", float("nan")), ("eps", -1.0),
                         ("weight_decay", -1.0), ("grad_scale", float("inf"))):
        bad = Z.zero_list_hparams([HP, HP])
        setattr(bad[1], field, value)
        word(lib.zero_list_adamw_step(ref(lst), bad, None), "hyper-parameters")
    bad = Z.zero_list_hparams([HP, dict(HP, step=2)])
    word(lib.zero_list_adamw8_step(ref(eight), bad, 0, None), "steps differ")
    for eps in (0.0, 9e-17):
        word(lib.zero_list_adamw8_step(ref(eight), Z.zero_list_hparams([HP, dict(HP, eps=eps)]), 0, None), "eps")
    word(lib.zero_list_adamw_step_dev(ref(lst), None, 16, None), "step state")
    word(lib.zero_list_adamw_step_dev(ref(lst), 16, 8, None), "group scalars")
    word(lib.zero_list_adamw8_step_dev(ref(eight), 24, 16, 0, None), "step state")
    word(lib.zero_list_adamw8_step_dev(ref(lst), 16, 16, 0, None), "fp32 state")
    need = Z.zero_list_grad_sqnorm_workspace_bytes(lst)
    word(lib.zero_list_grad_sqnorm(ref(lst), 256, need - 1, 16, 16, None), "workspace")
    word(lib.zero_list_grad_sqnorm(ref(lst), 264, need, 16, 16, None), "workspace")
    word(lib.zero_list_grad_sqnorm(ref(lst), 256, need, 12, 16, None), "misaligned")
    word(lib.zero_list_grad_sqnorm(ref(lst), 256, need, None, 16, None), "NULL")
    assert Z.zero_list_grad_sqnorm_workspace_bytes(Z.zero_list()) == 0
    word(lib.zero_list_decision_dev(16, 16, 1, 1.0, hp, 0, 16, 16, None), "n_groups")
    word(lib.zero_list_decision_dev(16, 16, 1, 1.0, hp, 65, 16, 16, None), "n_groups")
    word(lib.zero_list_decision_dev(16, 16, 0, 1.0, hp, 2, 16, 16, None), "n_ranks")
    word(lib.zero_list_decision_dev(None, 16, 1, 1.0, hp, 2, 16, 16, None), "NULL")
    word(lib.zero_list_decision_dev(16, 16, 1, 1.0, hp, 2, 8, 16, None), "step state")
    other, _ = planned([tensor(n=5001, layout=Z.ZERO_STATE_8BIT, m=None, v=None)])
    word(lib.zero_list_state8_pack(ref(lst), ref(other), None), "differ in size")
    word(lib.zero_list_state8_pack(ref(eight), ref(lst), None), "needs a list")
    word(lib.zero_list_state8_unpack(ref(eight), ref(eight), None), "needs a list")


def test_empty_lists_are_no_ops():
    hp = Z.zero_list_hparams([HP])
    for tensors in ([], [dict(numel=0)], [dict(numel=0, layout=Z.ZERO_STATE_8BIT)]):
        lst, _ = planned(tensors)
        if not tensors or tensors[0].get("layout"):
            Z.zero_list_adamw8_step(lst, hp, 1, stream=0)
        assert lst.update_blocks == lst.norm_blocks == lst.numel == 0


def test_binding_refuses_wrong_hparams_and_host_tensors():
    lst, _ = planned([tensor()], 2)
    with pytest.raises(ValueError, match="2 groups"):
        Z.zero_list_adamw_step(lst, Z.zero_list_hparams([HP]), stream=0)
    with pytest.raises(ValueError, match="GPU tensor"):
        Z.zero_list_plan([dict(numel=4, grad=torch.zeros(4, dtype=torch.bfloat16))])


# ---------------------------------------------------------------------- the plain forms


def test_reference_code_values():
    """e4m3 against torch's format of the same name; both tables strictly increasing from zero to their top."""
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.VALUES["m"], want, equal_nan=True)
    v = R.VALUES["v"]
    assert v[0] == 0 and v[1] == 2.0**-33 and v[255] == 1.875 and (np.diff(v) > 0).all()
    ratio = v[9:] / v[8:-1]
    assert ratio.max() == 1.125 and ratio.min() == 1.875**-1 * 2  # 6.7% to 12.5% apart


def test_reference_position_inverts_the_values():
    for which, last in (("m", 126), ("v", 255)):
        vals = R.VALUES[which][:last + 1].astype(np.float32)
        assert (R.position(vals, which) == np.arange(last + 1) << 20).all()
        mid = ((vals[1:].astype(np.float64) + vals[:-1]) / 2).astype(np.float32)
        assert (R.position(mid, which) == (np.arange(last) << 20) + (1 << 19)).all()


def test_reference_rounding_is_unbiased():
    """Every position between two codes, all 2^20 dithers at once: the mean code is the position, to 2^-20."""
    d = np.arange(1 << 20, dtype=np.int64)
    for frac in (0, 1, 12345, 1 << 19, (1 << 20) - 1):
        p = (37 << 20) + frac
        assert ((p + d) >> 20).mean() == pytest.approx(p / 2.0**20, abs=2.0**-21)


def test_reference_dither_is_uniform_over_seeds():
    """The dither of one element over 4096 seeds (and over steps): mean 1/2, standard error 1/sqrt(12·4096) = 0.0045;
    five of them allowed."""
    for j in (0, 255):
        for draws in ([R.dithers(s, 3, 7, 1) for s in range(4096)], [R.dithers(5, t, 7, 1) for t in range(4096)]):
            for k in (0, 1):
                assert abs(np.mean([d[k][0, j] for d in draws]) / 2.0**20 - 0.5) < 5 * 0.0045


def test_reference_update_in_fp32_against_64_bits():
    """Ten roundings of at most 2^-24 each reach m, v and the update; p adds the three of its own line."""
    rng = np.random.default_rng(1)
    n = 20000
    g, p, m = (rng.standard_normal(n) * s for s in (1e-3, 0.02, 3e-4))
    v = rng.random(n) * 1e-6 + 1e-9
    s = R.scalars(**HP, grad_scale=0.5, step=7)
    args = [x.astype(np.float32) for x in (g, p, m, v)]
    p32, m32, v32 = R.adamw(*args, s)
    p64, m64, v64 = R.adamw(*[a.astype(np.float64) for a in args], s, np.float64)
    u = 2.0**-24
    size_m = 0.9 * np.abs(args[2]) + 0.1 * 0.5 * np.abs(args[0])
    assert (np.abs(m32 - m64) <= 8 * u * size_m).all()
    assert (np.abs(v32 - v64) <= 10 * u * v64).all()
    step = s["step_size"] * size_m / (np.sqrt(v64) / s["bc2_sqrt"])
    assert (np.abs(p32 - p64) <= 4 * u * np.abs(args[1]) + 30 * u * step).all()


def test_conversion_between_two_gpus_is_refused():
    """The kernels read both lists' tables: a target on another GPU never reaches them (the lists here have no
    plan and no memory, only their devices)."""
    from mixed_precision_adam_amd.driver import TensorList

    a, b = TensorList.__new__(TensorList), TensorList.__new__(TensorList)
    a.device, b.device = torch.device("cuda", 0), torch.device("cuda", 1)
    a.list = b.list = Z.zero_list()
    for call in (a.pack8, a.unpack8, b.pack8):
        with pytest.raises(ValueError, match="one GPU"):
            call(b if call.__self__ is a else a)
