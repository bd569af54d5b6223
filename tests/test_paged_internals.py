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


@pytest.fixture(scope="module")
def collect(tmp_path_factory):
    """collect(words, failing read, failing clear) -> (error, expired, words after), with words in place of the device's."""
    lib = _compile(tmp_path_factory.mktemp("status"), "status", """
#include "kernels.h"
namespace {
int words[3], bad_read, bad_clear;
template <int I> binattn::StatusWord word() {
  return {[](int* v, cudaStream_t) { *v = words[I]; return I == bad_read ? cudaErrorUnknown : cudaSuccess; },
          [](cudaStream_t) { if (I == bad_clear) return cudaErrorUnknown; words[I] = 0; return cudaSuccess; }};
}
}
extern "C" int collect(int* w, int r, int c, int* expired) {
  for (int i = 0; i < 3; ++i) words[i] = w[i];
  bad_read = r; bad_clear = c;
  const binattn::StatusWord all[] = {word<0>(), word<1>(), word<2>()};
  bool x = false;
  const cudaError_t e = binattn::collect_status(all, 3, nullptr, &x);
  for (int i = 0; i < 3; ++i) w[i] = words[i];
  *expired = x;
  return e;
}
""")

    def call(words, bad_read=-1, bad_clear=-1):
        w, x = (ctypes.c_int * 3)(*words), ctypes.c_int()
        return lib.collect(w, bad_read, bad_clear, ctypes.byref(x)), bool(x.value), list(w)

    return call


def test_status_words_are_read_and_cleared(collect):
    assert collect([0, 0, 0]) == (0, False, [0, 0, 0])
    for words in ([1, 0, 0], [0, 1, 0], [0, 0, 1], [1, 1, 1]):
        assert collect(words) == (0, True, [0, 0, 0])


def test_an_error_loses_no_timeout(collect):
    """What a failing call does not return stays set for the next one."""
    for bad in range(3):
        err, _, left = collect([1, 1, 1], bad_read=bad)
        assert err != 0 and left == [1, 1, 1]
    assert collect([1, 0, 1], bad_clear=2) == (0, True, [0, 0, 1])
