"""The paged decode step's grid arithmetic, compiled for the host and called without a GPU."""
import ctypes
import os
import subprocess

import pytest

from sliding_window_recurrent_b200 import build as _build

SOURCE = """
#include "paged_grid.h"
extern "C" long long blocks(int B, int units, int max_pages, int page_size, int window, int teams, long long resident) {
  return maglev::decode_blocks(B, units, max_pages, page_size, window, teams, resident);
}
"""


@pytest.fixture(scope="module", params=["-O0", "-O2"])
def blocks(request, tmp_path_factory):
    d = tmp_path_factory.mktemp("grid")
    src, lib = d / "grid.cpp", d / "grid.so"
    src.write_text(SOURCE)
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", request.param, "-shared", "-fPIC", "-I" + _build.CSRC,
                    str(src), "-o", str(lib)], check=True)
    fn = ctypes.CDLL(str(lib)).blocks
    fn.restype = ctypes.c_longlong
    fn.argtypes = [ctypes.c_int] * 6 + [ctypes.c_longlong]
    return fn


def want(B, units, max_pages, page_size, window, teams, resident):
    """The same in unbounded integers: steps of 16 keys there can be at most, three more a unit, `teams` a block."""
    keys = max_pages * page_size
    if window:
        keys = min(keys, window + 16)
    return min(resident, -(-(-(-keys // 16) + 3) * units * B // teams))


@pytest.mark.parametrize("window", [0, 1, 15, 16, 512, 1 << 30, 2**31 - 17, 2**31 - 16, 2**31 - 15, 2**31 - 2, 2**31 - 1])
@pytest.mark.parametrize("B,units,max_pages,page_size", [
    (1, 1, 1, 16), (10, 10, 4, 16), (64, 10, 64, 64), (7, 65536, 1, 256), (1, 1, 1 << 26, 16), (32, 65536, 1 << 22, 256),
    (1 << 30, 1, 1, 16), (1 << 30, 65536, 1, 256)])
def test_the_grid_stays_between_one_block_and_what_is_resident(blocks, B, units, max_pages, page_size, window):
    """Every window the descriptor may hold, INT_MAX (no limit) among them: a grid beyond the resident blocks would
    number its teams past the workspace."""
    for teams, resident in ((1, 148 * 12), (4, 296), (4, 148), (12, 148)):
        got = blocks(B, units, max_pages, page_size, window, teams, resident)
        assert 1 <= got <= resident
        assert got == want(B, units, max_pages, page_size, window, teams, resident)
