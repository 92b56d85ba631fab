"""The host side of the list entry points under AddressSanitizer and UndefinedBehaviorSanitizer (CPU only; sanitizers
on the host compilation alone, the device code never runs)."""
import os

import pytest

from mixed_precision_adam_amd import build as B
from tests.test_host_sanitizers import NATIVE, ROOT, SAN, _run


def test_list_host_code_under_sanitizers(tmp_path):
    if not os.path.exists(B.HIPCC):
        pytest.skip("hipcc not available")
    flags = [f for f in B.FLAGS if f != "-O3"] + ["-O1", "-g"]
    host_san = [x for f in SAN for x in ("-Xarch_host", f)]
    objs = []
    for src in (B.SRC, B.LIST_SRC):
        objs.append(str(tmp_path / (os.path.basename(src) + ".o")))
        _run([B.HIPCC, *flags, *host_san, "-I", os.path.join(ROOT, "include"), "-c", "-o", objs[-1], src], tmp_path)
    exe = str(tmp_path / "list_host_checks")
    tlib = B.torch_lib_dir()
    _run([B.CLANG, "-std=c++17", "-O1", "-g", *SAN, "-I", os.path.join(ROOT, "include"), "-o", exe,
          os.path.join(NATIVE, "list_host_checks.cpp"), *objs, "-L", tlib, "-l:libamdhip64.so", f"-Wl,-rpath,{tlib}",
          "-lm"], tmp_path)
    assert "list host checks ok" in _run([exe], tmp_path)
