"""Host-callable parts of the library's sources, compiled by themselves (no GPU)."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_qk_attention_b200", "csrc")


def _compile(tmp, name, source):
    from bit_qk_attention_b200 import build
    src, out = tmp / f"{name}.cu", tmp / f"{name}.so"
    src.write_text(source)
    subprocess.run([build.NVCC, *build.ARCH, "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-I", CSRC, "-I",
                    os.path.join(ROOT, "include"), str(src), "-o", str(out)], check=True, capture_output=True)
    return ctypes.CDLL(str(out))


@pytest.fixture(scope="module")
def share_of(tmp_path_factory):
    f = _compile(tmp_path_factory.mktemp("share"), "share", """
#include "paged.cuh"
extern "C" int share(int64_t total, uint32_t ctas) { return binattn::share_of(total, ctas); }
""").share
    f.argtypes, f.restype = [ctypes.c_int64, ctypes.c_uint32], ctypes.c_int
    return f


def test_a_ctas_share_of_the_line(share_of):
    """Rounded up, also where the units and the grid together pass 32 bits."""
    for ctas in (1, 3, 148, 296, 444, 592):
        for total in (0, 1, ctas - 1, ctas, ctas + 1, 10**6, 2**31, 2**32 - ctas - 1, 2**32 - ctas, 2**32 - ctas + 1, 2**32 - 1,
                      2**32, 2**32 + 1, 2**38):
            want = -(-total // ctas)
            if want < 2**31:
                assert share_of(total, ctas) == want, (total, ctas)
