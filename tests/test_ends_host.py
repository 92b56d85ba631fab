"""The host side of the embedding, layer norm and loss head entry points (CPU only): sizes, the refusals of bad
arguments before anything is launched, calls that have nothing to do, and the binding's structure."""
import ctypes as C
import os
import shutil

import pytest
import torch

import mixed_precision_adam_amd as Z
from mixed_precision_adam_amd import driver
from tests.test_struct_layouts import ROOT, c_layout
from tests.test_struct_layouts import check as check_layout

LIB = Z.library()
BAD, OK = Z.ZERO_ERR_INVALID, Z.ZERO_OK
NAN, INF = float("nan"), float("inf")


def rows(n=4, cols=8, stride=None, dt=Z.ZERO_BF16, data=4096):
    return Z.zero_rows(data, n, cols, cols if stride is None else stride, dt, 0)


def refused(rc, *words):
    text = Z.zero_last_error()
    assert rc == BAD, (rc, text)
    assert all(w in text for w in words), text


def test_structure_matches_the_header(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    structs = {"zero_rows": Z.zero_rows}
    check_layout(c_layout(tmp_path, os.path.join(ROOT, "include"), "zero_shard.h", structs), structs)


# What no zero_rows may be, and a word of the message.
BAD_ROWS = [(dict(dt=3), "dtype"), (dict(dt=-1), "dtype"), (dict(n=-1), "out of range"),
            (dict(n=2**31), "out of range"), (dict(cols=0), "out of range"), (dict(cols=2**31), "out of range"),
            (dict(stride=7), "out of range"),
            (dict(stride=2**40), "out of range"), (dict(stride=-8), "out of range"), (dict(data=None), "no data"),
            (dict(data=4097), "aligned"), (dict(data=4098, dt=Z.ZERO_FP32), "aligned")]


@pytest.mark.parametrize("bad,word", BAD_ROWS)
def test_rows_are_checked_by_every_entry_point(bad, word):
    x, ids = rows(**bad), 8192
    good = rows(dt=bad.get("dt", Z.ZERO_BF16) if bad.get("dt") == Z.ZERO_FP32 else Z.ZERO_BF16)
    refused(LIB.zero_embed_forward(x, 0, ids, 8, 1.0, good, None), "table", word)
    refused(LIB.zero_embed_forward(good, 0, ids, 8, 1.0, x, None), "out", word)
    refused(LIB.zero_embed_grad(ids, 8, 0, x, 1.0, good, 0, 4096, 1 << 30, None), "out_grad", word)
    refused(LIB.zero_embed_grad(ids, 8, 0, good, 1.0, x, 0, 4096, 1 << 30, None), "table_grad", word)
    refused(LIB.zero_layernorm_forward(x, 4096, None, good.dt, 1e-5, 1, good, None, None, None), "x", word)
    refused(LIB.zero_layernorm_forward(good, 4096, None, good.dt, 1e-5, 1, x, None, None, None), "y", word)
    refused(LIB.zero_layernorm_grad(x, good, 4096, good.dt, 1, 4096, 4096, None, 4096, None, 2, 0, 4096, 1 << 30, None),
            "x", word)
    refused(LIB.zero_layernorm_grad(good, x, 4096, good.dt, 1, 4096, 4096, None, 4096, None, 2, 0, 4096, 1 << 30, None),
            "y_grad", word)
    refused(LIB.zero_layernorm_grad(good, good, 4096, good.dt, 1, 4096, 4096, x, 4096, None, 2, 0, 4096, 1 << 30, None),
            "x_grad", word)
    refused(LIB.zero_loss_head(x, good, ids, 8, 4096, 4096, 4096, 4096, 1 << 40, None), "x", word)
    refused(LIB.zero_loss_head(good, x, ids, 8, 4096, 4096, 4096, 4096, 1 << 40, None), "table", word)
    b = rows()
    if good.dt == Z.ZERO_BF16:
        refused(LIB.zero_loss_head_grad(b, b, ids, 8, 1.0, None, 4096, 4096, 4096, x, b, 0, 4096, 1 << 40, None),
                "x_grad", word)
        refused(LIB.zero_loss_head_grad(b, b, ids, 8, 1.0, None, 4096, 4096, 4096, b, x, 0, 4096, 1 << 40, None),
                "table_grad", word)


def test_rows_may_be_missing():
    refused(LIB.zero_embed_forward(None, 0, 8, 8, 1.0, rows(), None), "table is NULL")
    refused(LIB.zero_layernorm_forward(rows(), 16, None, 0, 1e-5, 1, None, None, None, None), "y is NULL")
    refused(LIB.zero_loss_head(rows(), None, 8, 8, 16, 16, 16, 4096, 1 << 40, None), "table is NULL")
    refused(LIB.zero_loss_head_grad(rows(), rows(), 8, 8, 1.0, None, 16, 16, 16, None, rows(), 0, 4096, 1 << 40, None),
            "x_grad is NULL")


def test_embedding_arguments():
    a, b = rows(), rows(3)
    refused(LIB.zero_embed_forward(a, -1, 8, 8, 1.0, b, None), "first_row")
    refused(LIB.zero_embed_forward(a, 0, 8, 2, 1.0, b, None), "ids of 2 bytes")
    refused(LIB.zero_embed_forward(a, 0, None, 8, 1.0, b, None), "no ids")
    refused(LIB.zero_embed_forward(a, 0, 4100, 8, 1.0, b, None), "ids misaligned")
    refused(LIB.zero_embed_forward(a, 0, 8, 8, 1.0, rows(3, 9), None), "cols")
    assert LIB.zero_embed_forward(a, 0, None, 8, 1.0, rows(0, data=None), None) == OK
    need = Z.zero_embed_grad_workspace_bytes(3, 4, 8)
    args = (8, 8, 0, b, 1.0, a, 0)
    refused(LIB.zero_embed_grad(*args, None, need, None), "workspace of 0 bytes")
    refused(LIB.zero_embed_grad(*args, 4096, need - 1, None), "workspace")
    refused(LIB.zero_embed_grad(*args, 4104, need, None), "16-byte aligned")
    refused(LIB.zero_embed_grad(8, 8, -1, b, 1.0, a, 0, 4096, need, None), "first_row")
    refused(LIB.zero_embed_grad(8, 8, 0, rows(3, 9), 1.0, a, 0, 4096, need, None), "cols")
    refused(LIB.zero_embed_grad(8, 3, 0, b, 1.0, a, 0, 4096, need, None), "ids of 3 bytes")
    assert LIB.zero_embed_grad(8, 8, 0, b, 1.0, rows(0, data=None), 0, 4096, need, None) == OK  # no table
    assert LIB.zero_embed_grad(None, 8, 0, rows(0, data=None), 1.0, a, 1, 4096, need, None) == OK  # nothing to add
    # a launch counts its threads in 32 bits: too many rows to fill, and too many column tiles
    refused(LIB.zero_embed_grad(8, 8, 0, rows(3), 1.0, rows(2**31 - 1), 0, 4096, 1 << 40, None), "one launch")
    wide = 1 << 21
    refused(LIB.zero_embed_grad(8, 8, 0, rows(2**18, wide), 1.0, rows(4, wide), 1, 4096, 1 << 50, None), "one launch")


def test_embedding_workspace():
    for n, table, cols in ((-1, 1, 1), (2**31, 1, 1), (1, -1, 1), (1, 2**31, 1), (1, 1, 0), (1, 1, 2**31)):
        assert Z.zero_embed_grad_workspace_bytes(n, table, cols) == 0
    for table, cols in ((1, 1), (50257, 1600), (16000, 5120), (2**20, 513)):
        sizes = [Z.zero_embed_grad_workspace_bytes(n, table, cols) for n in
                 (0, 1, 512, 513, 1000, 8192, 262_143, 262_144, 262_145, 300_000, 1 << 19, 1 << 22, (1 << 22) + 1)]
        assert sizes == sorted(sizes) and sizes[0] > 0, sizes  # what is made for n tokens does for fewer
    # 32 tokens a chunk, two fp32 edges of whole column tiles a chunk: an eighth of 16-bit rows
    assert Z.zero_embed_grad_workspace_bytes(8192, 50257, 1600) < 8192 * 2048 * 4 // 16 + (1 << 20)


def test_layernorm_arguments():
    x = rows()
    forward, grad = LIB.zero_layernorm_forward, LIB.zero_layernorm_grad
    refused(forward(x, None, None, 0, 1e-5, 1, x, None, None, None), "no weight")
    refused(forward(x, 16, None, 1, 1e-5, 1, x, None, None, None), "weight of dtype 1")
    refused(forward(x, 16, None, 7, 1e-5, 1, x, None, None, None), "weight of dtype 7")
    refused(forward(x, 17, None, 0, 1e-5, 1, x, None, None, None), "weight misaligned")
    refused(forward(x, 16, 18, 2, 1e-5, 1, x, None, None, None), "weight misaligned")
    for eps in (-1e-9, NAN, INF):
        refused(forward(x, 16, None, 0, eps, 1, x, None, None, None), "eps")
    refused(forward(x, 16, None, 0, 1e-5, 1, rows(5), None, None, None), "another shape")
    refused(forward(x, 16, None, 0, 1e-5, 1, rows(dt=1), None, None, None), "another shape or dtype")
    refused(forward(x, 16, None, 0, 1e-5, 1, x, 18, None, None), "statistics")
    refused(forward(x, 16, None, 0, 1e-5, 1, x, None, 18, None), "statistics")
    wide = rows(cols=Z.ZERO_LAYERNORM_MAX_COLS + 1)
    refused(forward(wide, 16, None, 0, 1e-5, 1, wide, None, None, None), "at most 16384")
    none = rows(0, data=None)
    assert forward(none, 16, None, 0, 1e-5, 1, none, None, None, None) == OK
    need = Z.zero_layernorm_grad_workspace_bytes(4, 8)
    refused(grad(x, x, 16, 0, 1, None, 16, x, 16, 16, 2, 0, 4096, need, None), "no statistics")
    refused(grad(x, x, 16, 0, 0, None, None, x, 16, 16, 2, 0, 4096, need, None), "no statistics")
    refused(grad(x, x, 16, 0, 1, 18, 16, x, 16, 16, 2, 0, 4096, need, None), "misaligned statistics")
    refused(grad(x, x, 16, 0, 1, 16, 16, x, 16, 16, 3, 0, 4096, need, None), "gradient dtype 3")
    refused(grad(x, x, 16, 0, 1, 16, 16, x, 18, 16, 2, 0, 4096, need, None), "gradient misaligned")
    refused(grad(x, x, 16, 0, 1, 16, 16, x, 16, 17, 0, 0, 4096, need, None), "gradient misaligned")
    refused(grad(x, rows(5), 16, 0, 1, 16, 16, x, 16, 16, 2, 0, 4096, need, None), "y_grad")
    refused(grad(x, x, 16, 0, 1, 16, 16, rows(5), 16, 16, 2, 0, 4096, need, None), "x_grad")
    refused(grad(x, x, 16, 0, 1, 16, 16, x, 16, 16, 2, 0, 4096, need - 1, None), "workspace")
    refused(grad(x, x, 16, 0, 1, 16, 16, x, 16, 16, 2, 0, None, need, None), "workspace of 0 bytes")
    assert grad(x, x, 16, 0, 1, 16, 16, None, None, None, 2, 0, 4096, need, None) == OK  # no result asked for
    assert grad(none, none, 16, 0, 1, None, None, none, 16, 16, 2, 1, 4096, need, None) == OK  # nothing to add
    assert Z.zero_layernorm_grad_workspace_bytes(1, 16385) == Z.zero_layernorm_grad_workspace_bytes(-1, 8) == 0
    most = Z.zero_layernorm_grad_workspace_bytes(2**31 - 1, 5120)
    assert 0 < Z.zero_layernorm_grad_workspace_bytes(1, 5120) < most <= 512 * 2 * 5120 * 4  # whatever the rows


def test_loss_head_arguments():
    x, w = rows(), rows(11)
    need = Z.zero_loss_head_workspace_bytes(4, 11, 8, False)
    out = (4096, 4096, 4096)
    head = LIB.zero_loss_head
    refused(head(rows(dt=2), rows(11, dt=2), 8, 8, *out, 4096, need, None), "16-bit")
    refused(head(x, rows(11, dt=1), 8, 8, *out, 4096, need, None), "16-bit")
    refused(head(x, rows(11, 9), 8, 8, *out, 4096, need, None), "cols")
    refused(head(x, rows(0, data=None), 8, 8, *out, 4096, need, None), "out of range")
    refused(head(x, rows((1 << 22) + 1), 8, 8, *out, 4096, 1 << 50, None), "out of range")
    refused(head(x, w, 8, 1, *out, 4096, need, None), "ids of 1 bytes")
    refused(head(x, w, None, 8, *out, 4096, need, None), "no ids")
    refused(head(x, w, 8, 8, None, 4096, 4096, 4096, need, None), "NULL output")
    refused(head(x, w, 8, 8, 4096, None, 4096, 4096, need, None), "NULL output")
    refused(head(x, w, 8, 8, 4096, 4096, None, 4096, need, None), "NULL output")
    refused(head(x, w, 8, 8, 4098, 4096, 4096, 4096, need, None), "misaligned output")
    refused(head(x, w, 8, 8, 4096, 4096, 4100, 4096, need, None), "misaligned output")
    refused(head(x, w, 8, 8, *out, 4096, need - 1, None), "workspace")
    refused(head(x, w, 8, 8, *out, 4096 + 16, need, None), "256-byte aligned")
    refused(head(x, w, 8, 8, *out, None, need, None), "workspace of 0 bytes")
    grad = LIB.zero_loss_head_grad
    need = Z.zero_loss_head_workspace_bytes(4, 11, 8)
    refused(grad(x, w, 8, 8, 1.0, None, *out, rows(5), w, 0, 4096, need, None), "x_grad has another shape")
    refused(grad(x, w, 8, 8, 1.0, None, *out, x, rows(11, dt=2), 0, 4096, need, None), "table_grad has another")
    for scale in (NAN, INF, -INF):
        refused(grad(x, w, 8, 8, scale, None, *out, x, w, 0, 4096, need, None), "scale")
    refused(grad(x, w, 8, 8, 1.0, 4100, *out, x, w, 0, 4096, need, None), "step state")
    refused(grad(x, w, 8, 8, 1.0, None, *out, x, w, 0, 4096, need - 1, None), "workspace")


def test_loss_head_workspace():
    for t, v, d in ((-1, 9, 8), (2**31, 9, 8), (4, 0, 8), (4, (1 << 22) + 1, 8), (4, 9, 0), (4, 9, (1 << 16) + 1),
                    (4, 1 << 22, 1 << 16)):
        assert Z.zero_loss_head_workspace_bytes(t, v, d) == 0
    for v, d in ((1, 1), (300, 40), (50257, 1600), (32000, 4096), (1 << 20, 64)):
        for gradients in (False, True):
            sizes = [Z.zero_loss_head_workspace_bytes(t, v, d, gradients) for t in
                     (0, 1, 256, 257, 1000, 2560, 2561, 4096, 8192, 100_000, 1 << 20)]
            assert sizes == sorted(sizes) and sizes[0] > 0, sizes
            if v > 30_000:  # past some thousands of tokens it stays as it is
                assert sizes[-1] == sizes[-3]
    # far below the fp32 scores of 65536 tokens and their softmax
    assert Z.zero_loss_head_workspace_bytes(65536, 50257, 1600) < 2 * 65536 * 50257 * 4 // 10


def test_the_binding_refuses_what_it_cannot_name():
    """Tensors that are not on a GPU, and what is no matrix of contiguous rows, are refused before any call."""
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU tensor"):
        Z.zero_embed_forward(x, torch.zeros(4, dtype=torch.int64), x)
    with pytest.raises(ValueError, match="int32 or int64"):
        Z._ids(torch.zeros(4), 4)
    with pytest.raises(ValueError, match="3 tokens for 4 rows"):
        Z._ids(torch.zeros(3, dtype=torch.int64), 4)
    with pytest.raises(ValueError, match="dtype"):
        Z._vector(torch.zeros(4, dtype=torch.float64), 4, "mean")
    with pytest.raises(ValueError, match="5 elements where 4"):
        Z._vector(torch.zeros(5), 4, "mean")
    with pytest.raises(ValueError, match="one value"):
        Z._scalar(torch.zeros(2), torch.float32, "loss")
    assert Z._vector(None, 4, "mean") == (None, None)
    r = rows()
    assert Z._rows(r) is r


class FakeGpu(torch.Tensor):
    """A tensor that says it is on a GPU: for the checks alone."""
    is_cuda = True


@pytest.mark.parametrize("make,word", [
    (lambda: torch.zeros(4, 8, 2), "matrix"), (lambda: torch.zeros(4, 8, dtype=torch.float64), "matrix"),
    (lambda: torch.zeros(8, 4).t(), "contiguous"), (lambda: torch.zeros(1, 8).expand(4, 8), "overlap"),
    (lambda: torch.zeros(40).as_strided((4, 8), (4, 1)), "overlap"), (lambda: torch.zeros(8), "matrix")])
def test_rows_of_a_tensor_are_checked(make, word):
    with pytest.raises(ValueError, match=word):
        Z._rows(make().as_subclass(FakeGpu))


def test_rows_of_a_tensor():
    for x, want in ((torch.zeros(4, 16)[:, :8], (4, 8, 16)), (torch.zeros(4, 1), (4, 1, 1)),
                    (torch.zeros(1, 8).expand(1, 8), (1, 8, 8)), (torch.zeros(0, 8), (0, 8, 8)),
                    (torch.zeros(6, 3)[:, 1:2], (6, 1, 3))):
        r = Z._rows(x.as_subclass(FakeGpu))
        assert (r.rows, r.cols, r.stride) == want and r.dt == Z.ZERO_FP32


def test_operators_check_what_they_are_made_of():
    with pytest.raises(ValueError, match="out of range"):
        driver.LossHead(torch.zeros(0, 8, dtype=torch.bfloat16), max_tokens=4)
    with pytest.raises(ValueError, match="out of range"):
        driver.LayerNorm(torch.zeros(16385))
    with pytest.raises(ValueError, match="out of range"):
        driver.TokenEmbedding(torch.zeros(4, 0), max_tokens=4)


@pytest.mark.parametrize("tokens", [0, 3])
def test_an_embedding_without_max_tokens_refuses_gradients(tokens):
    """It has no workspace, so not even the gradient of no tokens at all is taken."""
    table = torch.zeros(4, 8)
    op = driver.TokenEmbedding(table)
    op._on = lambda *tensors: None  # the tensors stand for ones on the operator's GPU
    with pytest.raises(ValueError, match="max_tokens"):
        op.grad(torch.zeros(tokens, dtype=torch.int64), torch.zeros(tokens, 8), table)


@pytest.mark.parametrize("vocab", [1, 300, 500, 4099, 50257])
@pytest.mark.parametrize("cols", [1, 64, 4096, 5120, 16384, 1 << 16])
def test_loss_head_workspace_is_bounded_whatever_the_tokens(vocab, cols):
    """A block of tokens is what it holds, so past a block it stays as it is, over small vocabularies too.  The bound
    adds up a block's parts at their most: codes and their turned copy (2^28 bytes each, or 256 tokens of them), 8 bytes
    an element of its hidden rows (2^30, or 256 tokens of them), the same again for parts of sums that are split (2^27)
    and small statistics (2^26), and the table's copies and sums (2 + 2 + 4 bytes an element)."""
    wide, words = -(-cols // 64) * 64, -(-vocab // 256) * 256
    codes, rows = max(1 << 28, 512 * words), max(1 << 30, 256 * 8 * wide)
    for gradients in (False, True):
        sizes = [Z.zero_loss_head_workspace_bytes(t, vocab, cols, gradients) for t in
                 (1, 256, 4096, 65536, 1 << 18, 1 << 20, 1 << 24, 2**31 - 1)]
        assert sizes == sorted(sizes) and sizes[-3] == sizes[-1], sizes
        assert sizes[-1] <= 2 * codes + rows + (1 << 27) + (1 << 26) + 8 * words * wide, sizes


@pytest.mark.parametrize("bad", [NAN, INF, -INF, 1e39, -1e39])
def test_factors_that_fp32_does_not_hold_are_refused(bad):
    """Times infinity, the zeros of a token outside the table and of a word without gradient would become NaN."""
    a, b = rows(), rows(3)
    refused(LIB.zero_embed_forward(a, 0, 8, 8, bad, b, None), "scale")
    refused(LIB.zero_embed_grad(8, 8, 0, b, bad, a, 0, 4096, Z.zero_embed_grad_workspace_bytes(3, 4, 8), None), "scale")
    refused(LIB.zero_loss_head_grad(b, a, 8, 8, bad, None, 4096, 4096, 4096, b, a, 0, 4096,
                                    Z.zero_loss_head_workspace_bytes(3, 4, 8), None), "scale")
    refused(LIB.zero_layernorm_forward(a, 16, None, 0, bad, 1, a, None, None, None), "eps")


def test_the_head_asks_for_a_copy_of_the_table_only_where_it_makes_one():
    need = Z.zero_loss_head_workspace_bytes_for
    for n in (0, 1, 33, 4096, 1 << 20):
        for gradients in (False, True):
            for v, d in ((50257, 1600), (32000, 4096), (300, 64)):
                most = Z.zero_loss_head_workspace_bytes(n, v, d, gradients)
                copy = -(-2 * v * d // 256) * 256
                for dt in (Z.ZERO_BF16, Z.ZERO_FP16):
                    assert need(n, rows(v, d, dt=dt), gradients) == most - copy
                    assert need(n, rows(v, d, d + 8, dt), gradients) == most - copy
                assert need(n, rows(v, d, d + 4), gradients) == most  # rows off the 16-byte lines
                assert need(n, rows(v, d, data=4096 + 8), gradients) == most
                assert need(n, rows(v, d, 1 << 22), gradients) == most
            assert need(n, rows(300, 65), gradients) == Z.zero_loss_head_workspace_bytes(n, 300, 65, gradients)
    assert need(4, rows(300, 64, dt=Z.ZERO_FP32)) == need(-1, rows(300, 64)) == need(4, rows(0, 64, data=None)) == 0
    # a call takes what was asked for, for its table and for as many tokens, and no less
    x, w = rows(4, 64), rows(11, 64)
    refused(LIB.zero_loss_head(x, w, 8, 8, 4096, 4096, 4096, 4096, need(4, w, False) - 1, None), "workspace")
    refused(LIB.zero_loss_head(x, rows(11, 64, 65), 8, 8, 4096, 4096, 4096, 4096, need(4, w, False), None), "workspace")
    refused(LIB.zero_loss_head_grad(x, w, 8, 8, 1.0, None, 4096, 4096, 4096, x, w, 0, 4096, need(4, w) - 1, None),
            "workspace")


def test_a_norm_without_gradients_holds_no_workspace():
    op = driver.LayerNorm(torch.ones(5120), gradients=False)
    assert op.ws is None and op.ws_bytes == 0
    with pytest.raises(ValueError, match="without gradients"):
        op.grad(torch.zeros(3, 5120), torch.zeros(3, 5120), torch.zeros(3), torch.zeros(3))
    with pytest.raises(ValueError, match="out of range"):
        driver.LayerNorm(torch.zeros(16385), gradients=False)
    assert driver.TokenEmbedding(torch.zeros(4, 8)).ws is None
    # what a norm with gradients holds, as its documentation says
    for cols, each in ((64, 16384), (1024, 16384), (1600, 4096), (16384, 4096)):
        assert Z.zero_layernorm_grad_workspace_bytes(2**31 - 1, cols) == each * cols
