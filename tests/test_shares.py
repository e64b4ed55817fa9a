"""How the shared decode's CTAs are shared out between its two lists: the same arithmetic that
the kernel does, compiled for the host."""
import ctypes
import os
import subprocess

import pytest

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "attention_fa_fwd_04_gb300", "csrc")
SOURCE = """#include "fa_shares.h"
extern "C" int ctas_of_tiles(long long a, long long z, long long starts, int ctas, int cost) {
  return fa::sh::ctas_of_tiles(a, z, starts, ctas, cost);
}
"""


@pytest.fixture(scope="module")
def ctas(tmp_path_factory):
    folder = tmp_path_factory.mktemp("shares")
    src, lib = folder / "shares.cpp", folder / "shares.so"
    src.write_text(SOURCE)
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I", CSRC, str(src), "-o", str(lib)])
    f = ctypes.CDLL(str(lib)).ctas_of_tiles
    f.argtypes = [ctypes.c_longlong] * 3 + [ctypes.c_int] * 2
    return f


@pytest.mark.parametrize("starts", [0, 2, 1024, 1 << 20])
@pytest.mark.parametrize("tiles", [1, 3, 9000, 1 << 40])
def test_nothing_streamed_leaves_all_ctas_to_the_tiles(ctas, tiles, starts):
    """Sequences of more than 16 rows have pieces, but no streamed list: all CTAs take tiles."""
    assert ctas(tiles, 0, starts, 152, 5) == 152


@pytest.mark.parametrize("starts", [0, 1, 1 << 20])
def test_no_tiles(ctas, starts):
    assert ctas(0, 77, starts, 152, 5) == 0
    assert ctas(0, 0, starts, 152, 5) == 0


@pytest.mark.parametrize("cost", [5, 6, 10])
def test_both_kinds_have_one_and_shares_go_by_cost(ctas, cost):
    for tiles in (1, 50, 3000, 1 << 33, 1 << 48):
        for streamed in (1, 40, 5000, 1 << 34, 1 << 48):
            for starts in (0, 30, 4096):
                n = ctas(tiles, streamed, starts, 152, cost)
                part = 16 * tiles * 152 // (16 * tiles + cost * (streamed + starts))
                assert n == min(151, max(1, part))
