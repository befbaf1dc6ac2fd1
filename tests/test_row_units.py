"""The units (CTAs or clusters) of the layer norm's kernels for any alignment and the
rows of partial sums that they write, whatever number of units the device holds at
once (CPU: csrc/row_units.h compiled for the host)."""
import ctypes
import os
import subprocess

import pytest

from gradient_quantization_gb300 import agoq

CSRC = os.path.join(agoq.HERE, "csrc")


@pytest.fixture(scope="module")
def units(tmp_path_factory):
    d = tmp_path_factory.mktemp("units")
    src, lib = d / "units.cpp", d / "units.so"
    src.write_text('#include "row_units.h"\n'
                   'extern "C" int partials(int64_t T, int64_t H) { return agoq::ln_partials(T, H); }\n'
                   'extern "C" int by_eights(int n, int64_t T, int most) '
                   '{ return agoq::by_eights(n, T, most); }\n')
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I" + CSRC, str(src),
                    "-o", str(lib)], check=True)
    L = ctypes.CDLL(str(lib))
    L.partials.argtypes = [ctypes.c_int64] * 2
    L.by_eights.argtypes = [ctypes.c_int, ctypes.c_int64, ctypes.c_int]
    return L


ROWS = list(range(1, 40)) + [303, 304, 305, 310, 2431, 2432, 2433, 1 << 20, (1 << 31) + 5, 1 << 40]
LENGTHS = [1, 5, 511, 512, 700, 1365, 2047, 2048, 4095, 4096, 5003, 39937]
RESIDENT = list(range(1, 20)) + [76, 152, 299, 304, 456, 1216]


def test_units_have_rows_and_partial_sums(units):
    """Every unit has a row, and a row of partial sums in the workspace; units that take more
    than one row keep their alignment (a multiple of eight rows apart)."""
    for T in ROWS:
        for H in LENGTHS:
            most = units.partials(T, H)
            assert 1 <= most <= T
            for n in RESIDENT:
                got = units.by_eights(min(n, T), T, most)
                assert 1 <= got <= most, (T, H, n, got)
                assert got == T or got % 8 == 0, (T, H, n, got)


def test_workspace_holds_the_partial_sums(units):
    wb = agoq.lib().agoq_layernorm_backward_workspace_bytes
    for T in (1, 3, 7, 8, 100, 1 << 20):
        for H in LENGTHS:
            assert wb(T, H) == units.partials(T, H) * 2 * H * 4


def test_as_many_as_are_resident(units):
    """Whole devices: the units that are resident, rounded to eights where they take several
    rows."""
    assert units.by_eights(456, 6151, 1 << 20) == 456
    assert units.by_eights(300, 6151, 304) == 296
    assert units.by_eights(304, 6151, 304) == 304
    assert units.by_eights(5, 5, 5) == 5 and units.by_eights(9, 9, 9) == 9
