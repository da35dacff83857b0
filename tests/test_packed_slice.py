"""The rows of a sequence between two entries of cu_seqlens, whatever they hold:
the kernels' own arithmetic, compiled for the host (no GPU)."""
import ctypes
import itertools
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "variable_length_prefill_gb300", "csrc")
LEAST, MOST = -2 ** 31, 2 ** 31 - 1


@pytest.fixture(scope="module")
def slice_of(tmp_path_factory):
    cxx = shutil.which("g++") or pytest.skip("no g++")
    at = tmp_path_factory.mktemp("slice")
    (at / "s.cc").write_text('#include "packed_slice.h"\n'
                             'extern "C" long long f(int a, int b, int t) {\n'
                             '  avp::PackedSlice s = avp::packed_slice(a, b, t);\n'
                             '  return (long long)s.lo << 32 | (unsigned)s.n;\n}\n')
    subprocess.run([cxx, "-std=c++17", "-O1", "-fsanitize=signed-integer-overflow",
                    "-fno-sanitize-recover=all", "-static-libubsan", "-shared", "-fPIC", "-I", CSRC,
                    str(at / "s.cc"), "-o", str(at / "s.so")], check=True, capture_output=True)
    f = ctypes.CDLL(str(at / "s.so")).f
    f.restype, f.argtypes = ctypes.c_longlong, [ctypes.c_int] * 3
    return lambda a, b, t: (f(a, b, t) >> 32, f(a, b, t) & 0xFFFFFFFF)


def test_any_entries(slice_of):
    ends = [LEAST, LEAST + 1, LEAST + 7, -2 ** 30, -5, -1, 0, 1, 5, 8, 9, 100, 2 ** 30, MOST - 1, MOST]
    for a, b, total in itertools.product(ends, ends, [0, 1, 8, 100, MOST]):
        lo, n = slice_of(a, b, total)
        rows = [max(0, min(x, total)) for x in (a, b)]
        assert n == max(0, rows[1] - rows[0]), (a, b, total)
        assert 0 <= lo <= lo + n <= total and (n == 0 or lo == rows[0]), (a, b, total)


@pytest.mark.parametrize("name", ["paged_cache.cu", "paged_tree.cu"])
def test_kernels_use_it(name):
    """No kernel of the paged operators subtracts entries of cu_seqlens itself."""
    with open(os.path.join(CSRC, name)) as f:
        src = f.read()
    uses = [line for line in src.splitlines() if re.search(r"__ldg\((p\.)?cu \+", line)]
    assert uses and all("packed_slice(" in line for line in uses), uses
