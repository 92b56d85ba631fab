"""The kernels of the embedding, layer norm and loss head entry points on the CPU, under AddressSanitizer and
UndefinedBehaviorSanitizer: tests/native/lockstep/ runs the library's own sources with every thread of a workgroup as a
fiber, over buffers of exactly the sizes that a call may touch, and compares the results with sums in 64 bits.  The host
side of the entry points (sizes, checks, launches) runs with them."""
import concurrent.futures
import os
import platform

import pytest

from mixed_precision_adam_amd import build as B
from tests.test_host_sanitizers import NATIVE, ROOT, SAN, _run


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    if not os.path.exists(B.CLANG) or platform.machine() != "x86_64":
        pytest.skip("clang for x86-64 is needed")
    folder = tmp_path_factory.mktemp("lockstep")
    flags = ["-x", "c++", "-std=c++17", "-O2", "-g", *SAN, "-I", os.path.join(NATIVE, "lockstep"), "-I",
             os.path.join(ROOT, "include"), "-c"]
    sources = (B.EMBED_SRC, B.NORM_SRC, B.HEAD_SRC, os.path.join(NATIVE, "ends_kernel_checks.cpp"))
    objs = [str(folder / (os.path.basename(src) + ".o")) for src in sources]
    with concurrent.futures.ThreadPoolExecutor(len(sources)) as pool:
        list(pool.map(lambda src, obj: _run([B.CLANG, *flags, "-o", obj, src], folder), sources, objs))
    exe = str(folder / "ends_kernel_checks")
    _run([B.CLANG, *SAN, "-o", exe, *objs], folder)
    return exe


@pytest.mark.parametrize("part", ["embedding", "norm", "head"])
def test_kernels_under_sanitizers(program, part, tmp_path):
    assert "kernel checks ok" in _run([program, part], tmp_path)
