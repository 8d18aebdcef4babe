"""Tables of sequence offsets of any content (CPU only): the runs that the linear
recurrence's waves find in them, compiled for the host."""
import ctypes
import os
import random
import subprocess

import pytest

from gated_deltanet_chunked_rule_amd import build

RUNS = r"""
#include "gdr_layer.h"
extern "C" int runs(const int32_t* cu, int N, int T, int Ttot, int t0, int count, uint32_t* out) {
  gdr::SeqFinder f;
  f.cu = cu; f.N = N; f.T = T; f.Ttot = Ttot; f.packed = cu != nullptr;
  int seq[32];
  for (int& n : seq) n = -1;
  const gdr::TokenRuns m = gdr::token_runs(f, t0, count, seq);
  out[0] = m.first; out[1] = m.last; out[2] = m.gap;
  for (int k = 0; k < 32; ++k) {   // what a run's ends index: a row of the states
    if (k < count && ((m.first | m.last) >> k & 1)) {
      if (t0 + k >= Ttot) return 1;
      if (seq[k] < 0 || seq[k] >= N) return 2;
      if (cu && f.at(seq[k]) > t0 + k) return 3;
      if (!cu && seq[k] != (t0 + k) / T) return 4;
    } else if (seq[k] != -1) {
      return 5;
    }
  }
  for (int k = 0; k < count; ++k) out[3 + k] = (uint32_t)seq[k];
  return 0;
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    at = tmp_path_factory.mktemp("runs")
    src, out = at / "runs.cpp", at / "runs.so"
    src.write_text(RUNS)
    subprocess.run([build.hipcc(), "-x", "hip", "--offload-host-only", "-O1", "-std=c++17", "-fPIC", "-shared", "-I", build.CSRC,
                    "-I", os.path.join(build.ROOT, "include"), str(src), "-o", str(out)], check=True)
    return ctypes.CDLL(str(out))


def runs(lib, cu, N, T, total, t0, count):
    table, out = None if cu is None else (ctypes.c_int32 * len(cu))(*cu), (ctypes.c_uint32 * 38)()
    assert lib.runs(table, N, T, total, t0, count, out) == 0, (cu, total, t0)
    first, last, gap = out[:3]
    mask = (1 << count) - 1
    assert first & gap == 0 and (first | last) & ~mask == 0
    assert t0 > 0 or count == 0 or (first | gap) & 1      # token 0 goes on from nothing
    return first, last, gap & mask, out[3:3 + count]


def test_any_table_stays_inside_the_buffers(lib):
    rng = random.Random(5)
    for _ in range(20000):
        T, count = rng.choice([0, 1, 5, 64, 65, 130]), rng.choice([4, 8, 16])
        value = rng.choice([lambda: rng.randint(0, T), lambda: rng.randint(-T - 1, 2 * T + 1), lambda: rng.choice([-2 ** 31, 2 ** 31 - 1, 0, T])])
        cu = [value() for _ in range(rng.randint(2, 9))]
        for t0 in range(0, max(T, 1) + 2 * count, count):
            runs(lib, cu, len(cu) - 1, 0, T, t0, count)


@pytest.mark.parametrize("count", [4, 8, 16])
def test_tables_that_do_not_decrease(lib, count):
    rng = random.Random(6)
    for _ in range(2000):
        T = rng.choice([1, 63, 64, 130])
        if rng.random() < 0.3:
            B = rng.randint(1, 4)
            cu, table, total = [T * b for b in range(B + 1)], None, T * B
        else:
            cu, total = sorted(rng.randint(0, T) for _ in range(rng.randint(2, 9))), T
            table = cu
        for t0 in range(0, total, count):
            first, last, gap, seq = runs(lib, table, len(cu) - 1, T, total, t0, count)
            for k in range(count):
                t, bit = t0 + k, lambda m: m >> k & 1
                inside = any(a <= t < b for a, b in zip(cu, cu[1:]))
                starts = any(a == t < b for a, b in zip(cu, cu[1:]))
                ends = any(a <= t == b - 1 for a, b in zip(cu, cu[1:]))
                if starts or ends:
                    assert cu[seq[k]] <= t < cu[seq[k] + 1]
                assert (bit(first), bit(last), bit(gap)) == (starts, ends, not inside), (cu, t0, k)
