"""CTAs that share the K of a tile of the FP4 product (CPU: csrc/fp4_split.h compiled for the host):
each has stages of 256 elements."""
import ctypes
import os
import subprocess

import pytest

from gradient_quantization_gb300 import agoq

CSRC = os.path.join(agoq.HERE, "csrc")


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    d = tmp_path_factory.mktemp("split")
    src, lib = d / "split.cpp", d / "split.so"
    src.write_text('#include "fp4_split.h"\n'
                   'extern "C" int few_rows(int64_t s, int64_t t, int n) { return agoq::fp4_split_few_rows(s, t, n); }\n'
                   'extern "C" int few_tiles(int64_t s, int64_t t, int n) { return agoq::fp4_split_few_tiles(s, t, n); }\n')
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I" + CSRC, str(src),
                    "-o", str(lib)], check=True)
    L = ctypes.CDLL(str(lib))
    for f in (L.few_rows, L.few_tiles):
        f.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int]
    return L


STAGES = list(range(1, 300)) + [1000, 4095, 65535, 65536]
TILES = list(range(1, 310)) + [1000, 1 << 23]


@pytest.mark.parametrize("sms", [152, 148, 20])
def test_every_cta_has_stages(rule, sms):
    for stages in STAGES:
        for tiles in TILES:
            c = rule.few_rows(stages, tiles, sms)
            assert 1 <= c <= 8 and (c == 1 or c * tiles <= 2 * sms), (stages, tiles, c)
            assert (c - 1) * -(-stages // c) < stages, (stages, tiles, c)
            c = rule.few_tiles(stages, tiles, sms)
            assert 0 <= c <= 8 and c * tiles <= sms, (stages, tiles, c)
            if c:
                assert (c - 1) * -(-stages // c) < stages, (stages, tiles, c)


def test_choices(rule):
    """Sizes of the comments, and ones of which a CTA would have had nothing."""
    assert [rule.few_rows(16, t, 152) for t in (86, 32, 300, 400)] == [3, 4, 1, 1]
    assert [rule.few_rows(s, 4, 152) for s in (1, 4, 5, 6, 9, 33, 64)] == [1, 4, 3, 3, 3, 7, 8]
    assert rule.few_rows(4, 80, 152) == 2
    assert rule.few_tiles(36, 6, 152) == 4 and rule.few_tiles(16, 16, 152) == 2
