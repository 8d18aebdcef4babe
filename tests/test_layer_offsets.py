"""Tables of sequence offsets of any content (CPU only): the kernels' own lookup,
compiled for the host, walked as the convolution and the scan walk it."""
import ctypes
import os
import random
import subprocess

import pytest

from gated_deltanet_chunked_rule_amd import build

WALK = r"""
#include "gdr_layer.h"
using gdr::SeqFinder;
static SeqFinder finder(const int32_t* cu, int N, int Ttot) {
  SeqFinder f;
  f.cu = cu; f.N = N; f.T = 0; f.Ttot = Ttot; f.packed = true;
  return f;
}
// The scan's output pass over segments of `seg` tokens.  0, or the number of the first rule that does not hold.
// from[t] = 1 + n where the run at t starts from sequence n's initial state, -s where it starts from the state that
// another workgroup leaves at the end of segment s - 1, INT32_MIN where it belongs to no sequence; 0 inside a run.
extern "C" int walk(const int32_t* cu, int N, int Ttot, int seg, int32_t* from) {
  const SeqFinder f = finder(cu, N, Ttot);
  const int segs = (Ttot + seg - 1) / seg;
  for (int s = 0; s < segs; ++s) {
    const int seg0 = s * seg, seg1 = seg0 + seg < Ttot ? seg0 + seg : Ttot;
    for (int t = seg0; t < seg1;) {
      int start, end;
      const int n = f.find(t, start, end);
      if (end <= t || end > Ttot || n >= N || n < -1) return 1;
      const int stop = end < seg1 ? end : seg1;
      if (n < 0) {
        from[t] = INT32_MIN;
      } else {
        if (start < 0 || start > t) return 2;
        const bool on = SeqFinder::goes_on(t, seg0, start);
        if (on && s == 0) return 3;
        from[t] = on ? -s : 1 + n;
      }
      for (int i = t + 1; i < stop; ++i) from[i] = 0;
      t = stop;
    }
  }
  return 0;
}
// The rows that the convolution reads around tokens and ends of sequences, W taps.
extern "C" int taps(const int32_t* cu, int N, int Ttot, int W) {
  const SeqFinder f = finder(cu, N, Ttot);
  auto row = [&](int start, int t, int end) {   // an input row of [0, end), or a row of the initial state
    if (t >= start) return t >= 0 && t < end && end <= Ttot;
    return W - 1 + t - start >= 0 && W - 1 + t - start < W - 1;
  };
  for (int t = 0; t < Ttot; ++t) {
    int start, end;
    if (f.find(t, start, end) < 0) continue;
    for (int j = 0; j < W; ++j)
      if (!row(start, t - (W - 1) + j, end)) return 1;
    if (t >= end - (W - 1) && t - (end - (W - 1)) >= W - 1) return 2;   // row of the final state's gradient
  }
  for (int n = 0; n < N; ++n) {
    const int start = f.at(n), end = f.at(n + 1) > start ? f.at(n + 1) : start;
    if (start < 0 || end > Ttot) return 3;
    for (int i = 0; i < W - 1; ++i)
      if (!row(start, end - (W - 1) + i, end)) return 4;
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    at = tmp_path_factory.mktemp("offsets")
    src, out = at / "walk.cpp", at / "walk.so"
    src.write_text(WALK)
    subprocess.run([build.hipcc(), "-x", "hip", "--offload-host-only", "-O1", "-std=c++17", "-fPIC", "-shared", "-I", build.CSRC,
                    "-I", os.path.join(build.ROOT, "include"), str(src), "-o", str(out)], check=True)
    return ctypes.CDLL(str(out))


def walk(lib, cu, T, seg):
    table, out = (ctypes.c_int32 * len(cu))(*cu), (ctypes.c_int32 * max(T, 1))()
    assert lib.walk(table, len(cu) - 1, T, seg, out) == 0, (cu, T, seg)
    for W in (2, 3, 4):
        assert lib.taps(table, len(cu) - 1, T, W) == 0, (cu, T, W)
    return list(out)[:T]


def test_a_decreasing_table_starts_from_a_state_that_exists(lib):
    # at token 10 the table names a run that starts at 5: no segment stands before the first one
    assert walk(lib, [0, 10, 5, 20], 20, 64)[10] == 1 + 2
    # nor is token 70 the first of its segment
    got = walk(lib, [0, 70, 30, 150], 150, 64)
    assert got[64] == -1 and got[70] == 1 + 2 and got[128] == -2


def test_any_table_stays_inside_the_buffers(lib):
    rng = random.Random(5)
    for _ in range(20000):
        T = rng.choice([1, 5, 64, 65, 130, 300])
        value = rng.choice([lambda: rng.randint(0, T), lambda: rng.randint(-T, 2 * T), lambda: rng.choice([-2 ** 31, 2 ** 31 - 1, 0, T, rng.randint(0, T)])])
        walk(lib, [value() for _ in range(rng.randint(2, 9))], T, rng.choice([64, 128]))


def test_tables_that_do_not_decrease_carry_every_state(lib):
    rng = random.Random(6)
    for _ in range(5000):
        T, seg = rng.choice([1, 64, 130, 300, 700]), rng.choice([64, 128])
        cu = sorted(rng.randint(0, T) for _ in range(rng.randint(2, 9)))
        got = walk(lib, cu, T, seg)
        for t in range(T):
            n = max((i for i in range(len(cu) - 1) if cu[i] <= t < cu[i + 1]), default=None)
            if n is None:
                assert got[t] in (0, -2 ** 31)
            elif t == cu[n]:
                assert got[t] == 1 + n
            elif t % seg == 0:
                assert got[t] == -(t // seg)
            else:
                assert got[t] == 0
