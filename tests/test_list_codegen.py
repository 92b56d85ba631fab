"""Code generation of the list kernels (CPU only: compiles the source to gfx950 assembly with the library's own flags).

* Every wide vector access carries the non-temporal hint: each byte is used once.
* Accesses through descriptor addresses are global, not flat, and nothing spills to scratch memory.
* The rules on scalar memory and packed arithmetic that hold for the library's other source."""
import os
import re
import subprocess

import pytest

from mixed_precision_adam_amd import build as B
from tests import test_codegen


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    if not os.path.exists(B.HIPCC):
        pytest.skip("hipcc not available")
    out = str(tmp_path_factory.mktemp("asm") / "list.s")
    flags = [f for f in B.FLAGS if f != "-fPIC"]
    subprocess.run([B.HIPCC, *flags, "-I", os.path.join(B.ROOT, "include"), "--cuda-device-only", "-S", "-o", out,
                    B.LIST_SRC], check=True, capture_output=True)
    return open(out).read()


def test_wide_accesses_are_nontemporal_and_global(asm):
    ks = test_codegen.kernels(asm)
    found = {k: [b for n, b in ks.items() if k in n] for k in ("list_sqnorm_kernel", "list_adamw_kernel",
                                                                "list_adamw8_kernel", "list_pack8_kernel",
                                                                "list_unpack8_kernel", "list_unpack8_moments_kernel")}
    assert [len(v) for v in found.values()] == [1, 1, 1, 1, 1, 1]
    for kernel, bodies in found.items():
        for body in bodies:
            assert not [x for x in body if re.match(r"(flat|scratch)_", x)], kernel
            wide = [x for x in body if re.match(r"global_(load|store)_dwordx[24]\b", x)]
            plain = [x for x in wide if not re.search(r"\bnt\b", x)]
            others = 1 if kernel == "list_sqnorm_kernel" else 0  # the partial sum's store
            assert len(wide) >= 4 and len(plain) <= others, f"{kernel}: {plain[:3]}"


def test_no_scalar_memory_writes_and_no_packed_fp32(asm):
    test_codegen.test_no_scalar_memory_writes_and_no_packed_fp32(asm)
