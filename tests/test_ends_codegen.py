"""Code generation of the embedding, layer norm and loss head kernels (CPU only: compiles the sources to gfx950 assembly
with the library's own flags).

* Memory accesses are global, not flat, and nothing spills to scratch memory.
* Units move in 16-byte accesses; the products load straight into LDS and multiply on the matrix cores, and wait for
  loads only where a step meets; they keep everything in registers.
* The rules on scalar memory and packed arithmetic that hold for the library's other sources."""
import os
import re
import subprocess

import pytest

from mixed_precision_adam_amd import build as B
from tests import test_codegen

SOURCES = {"embed": B.EMBED_SRC, "norm": B.NORM_SRC, "head": B.HEAD_SRC}


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    if not os.path.exists(B.HIPCC):
        pytest.skip("hipcc not available")
    folder = tmp_path_factory.mktemp("asm")
    flags = [f for f in B.FLAGS if f != "-fPIC"]
    runs = {}
    for name, src in SOURCES.items():
        out = str(folder / f"{name}.s")
        runs[out] = name, subprocess.Popen([B.HIPCC, *flags, "-I", os.path.join(B.ROOT, "include"),
                                            "--cuda-device-only", "-S", "-o", out, src], stderr=subprocess.DEVNULL)
    for _, p in runs.values():
        assert p.wait() == 0
    return {name: open(out).read() for out, (name, _) in runs.items()}


@pytest.mark.parametrize("source", SOURCES)
def test_no_flat_accesses(asm, source):
    for name, body in test_codegen.kernels(asm[source]).items():
        assert "sort_pass_kernel" in name or not [x for x in body if x.startswith("flat_")], name


@pytest.mark.parametrize("source,kernel", [("embed", "embed_forward_kernel"), ("embed", "embed_grad_few_kernel"),
                                           ("embed", "embed_grad_kernel"), ("norm", "layernorm_forward_kernel"),
                                           ("norm", "layernorm_grad_kernel")])
def test_units_move_in_16_bytes(asm, source, kernel):
    found = [(n, b) for n, b in test_codegen.kernels(asm[source]).items() if kernel in n]
    assert found
    for name, body in found:
        for access in ("load", "store"):
            assert [x for x in body if re.match(rf"global_{access}_dwordx4\b", x)], (name, access)


def test_products_run_on_the_matrix_cores(asm):
    found = {n: b for n, b in test_codegen.kernels(asm["head"]).items()
             if re.search(r"(scores|x_grad|table_grad)_kernel", n)}
    assert len(found) == 6  # three products, two formats
    for name, body in found.items():
        assert not [x for x in body if x.startswith("scratch_")], name
        kind = "bf16" if "ILi0E" in name else "f16"
        assert sum(x.startswith(f"v_mfma_f32_16x16x32_{kind}") for x in body) >= 128, name
        assert [x for x in body if re.match(r"buffer_load_dwordx4 .* lds$", x)], name
        # in the loop: a wait for loads directly before a barrier, and nowhere else
        first, last = (f(k for k, x in enumerate(body) if x.startswith("v_mfma")) for f in (min, max))
        loop = body[first:last]
        for k, x in enumerate(loop):
            if x.startswith("s_waitcnt") and "vmcnt" in x:
                assert any(y.startswith("s_barrier") for y in loop[k:k + 4]), (name, loop[k:k + 4])


@pytest.mark.parametrize("source", SOURCES)
def test_no_scalar_memory_writes_and_no_packed_fp32(asm, source):
    test_codegen.test_no_scalar_memory_writes_and_no_packed_fp32(asm[source])


RAGGED_8_UNITS = re.compile(r"layernorm_grad_kernelILi\dELi8ELi4ELb1E")


def scratch(body):
    return [x for x in body if x.startswith("scratch_")]


@pytest.mark.parametrize("source", SOURCES)
def test_stores_do_not_go_through_scratch_memory(asm, source):
    """Units stay in registers up to their store, whole rows and ragged ones."""
    for name, body in test_codegen.kernels(asm[source]).items():
        assert RAGGED_8_UNITS.search(name) or not scratch(body), (name, scratch(body)[:3])


def test_ragged_rows_of_eight_units_a_lane_stay_in_registers(asm):
    """Layer norm's backward pass over 8193 to 16384 ragged columns: the widest form, in each format."""
    found = {n: b for n, b in test_codegen.kernels(asm["norm"]).items() if RAGGED_8_UNITS.search(n)}
    assert len(found) == 3
    for name, body in found.items():
        assert not scratch(body), (name, len(scratch(body)))


def test_the_sort_reads_and_writes_its_places_as_lds(asm):
    """No flat access in a pass of the sort either: each would wait for the wavefront's global stores and atomics."""
    found = [b for n, b in test_codegen.kernels(asm["embed"]).items() if "sort_pass_kernel" in n]
    assert len(found) == 1 and not [x for x in found[0] if x.startswith("flat_")]
    assert [x for x in found[0] if x.startswith("ds_write_b32")]


def unwaited_barriers(text):
    """Barriers of a kernel that loads into LDS may pass before they have landed, over all its barriers from the first
    such load on.  Going back from a barrier there has to be a wait for all loads before any load into LDS, and before
    any label or branch, past which another way may lead to the barrier."""
    lines = [x.split(";")[0].strip() for x in text.splitlines()]
    lines = [x for x in lines if x]
    loads = [k for k, x in enumerate(lines) if re.match(r"buffer_load_\w+ .* lds$", x)]
    barriers = [k for k, x in enumerate(lines) if x.startswith("s_barrier") and loads and k > loads[0]]
    bad = []
    for k in barriers:
        for x in reversed(lines[:k]):
            if re.match(r"s_waitcnt .*\bvmcnt\(0\)", x):
                break
            if x.endswith(":") or re.match(r"(s_c?branch|s_barrier|buffer_load_\w+ .* lds$)", x):
                bad.append(k)
                break
    return barriers, bad


def test_staged_data_has_landed_at_every_barrier_of_the_products(asm):
    text = asm["head"]
    found = 0
    for m in re.finditer(r"^(_Z\S*(?:scores|x_grad|table_grad)_kernel\S*):\s*;\s*@", text, re.M):
        body = text[m.end():text.index(".Lfunc_end", m.end())]
        barriers, bad = unwaited_barriers(body)
        assert len(barriers) >= 2 and not bad, (m.group(1), len(barriers), bad)
        # the check sees a wait that is missing, at either barrier of the loop
        waits = [w for w in re.finditer(r"\bvmcnt\(0\)", body)]
        assert waits
        for w in waits:
            without = body[:w.start()] + "vmcnt(5)" + body[w.end():]
            before = body[:w.start()].count("\n")
            if re.search(r"^\s*s_barrier", "\n".join(body.splitlines()[before:before + 4]), re.M):
                assert unwaited_barriers(without)[1], (m.group(1), before)
        found += 1
    assert found == 6


def test_the_products_ask_for_the_wait_themselves():
    """Whatever the compiler makes of a barrier: no bare one stands in the source of the staged loop."""
    source = open(B.HEAD_SRC).read()
    tile = source[source.index("struct Tile {"):source.index("// Which tile and split")]
    assert tile.count("meet();") == 2 and "__syncthreads" not in tile
    assert re.search(r"void meet\(\) \{\s*__builtin_amdgcn_s_waitcnt\(0x0F70\);[^\n]*\n\s*__syncthreads\(\);", source)
