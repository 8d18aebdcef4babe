"""Which channel each value of a column of the linear recurrence stands for (CPU
only, compiled for the host): one that is there, and the one that its lane holds."""
import ctypes
import os
import subprocess

import pytest

from gated_deltanet_chunked_rule_amd import build

COLUMNS = r"""
#include "gdr_layer.h"
extern "C" int width() { return gdr::kLinCh; }
extern "C" int lanes() { return gdr::kLinCh / gdr::kLinVec; }
extern "C" int channel(int col, int c, int D) { return gdr::lin_channel(col, c, D); }
// the first channel of the lane that holds value c, and c's place there
extern "C" int base(int col, int c, int D) { return gdr::lin_base(col * gdr::kLinCh + c / gdr::kLinVec * gdr::kLinVec, D); }
extern "C" int place(int c, int D) { return gdr::lin_place(c, D); }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    at = tmp_path_factory.mktemp("columns")
    src, out = at / "columns.cpp", at / "columns.so"
    src.write_text(COLUMNS)
    subprocess.run([build.hipcc(), "-x", "hip", "--offload-host-only", "-O1", "-std=c++17", "-fPIC", "-shared", "-I", build.CSRC,
                    "-I", os.path.join(build.ROOT, "include"), str(src), "-o", str(out)], check=True)
    return ctypes.CDLL(str(out))


@pytest.mark.parametrize("D", [1, 2, 3, 4, 63, 64, 65, 127, 128, 129, 130, 255, 256, 257, 513, 2 ** 25 - 1, 2 ** 25])
def test_every_value_is_a_channel_that_its_lane_holds(lib, D):
    width, cols = lib.width(), -(-D // lib.width())
    for col in {0, cols // 2, max(0, cols - 2), cols - 1}:
        seen = set()
        for c in range(width):
            d = lib.channel(col, c, D)
            assert 0 <= d < D, (col, c, d)          # a word of the next tile otherwise
            assert d == lib.base(col, c, D) + lib.place(c, D) and 0 <= lib.place(c, D) < min(D, width // lib.lanes())
            seen.add(d)
        assert seen >= set(range(col * width, min(D, (col + 1) * width)))
