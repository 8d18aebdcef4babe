"""Sequences without a token, and sequence numbers at the end of an int (CPU only,
compiled for the host): walked once each, by shares that end."""
import ctypes
import os
import random
import subprocess

import pytest

from gated_deltanet_chunked_rule_amd import build

SEQUENCES = r"""
#include <sys/mman.h>
#include "gdr_layer.h"
static gdr::SeqFinder finder(const int32_t* cu, int N, int T, int Ttot) {
  gdr::SeqFinder f;
  f.cu = cu; f.N = N; f.T = T; f.Ttot = Ttot; f.packed = cu != nullptr;
  return f;
}
// counts[n] is raised for every n met, up to `most` of them; how many
extern "C" long met(const int32_t* cu, int N, int T, int Ttot, long first, long step, long most, long* at) {
  long k = 0;
  struct Enough {};
  try {
    gdr::empty_sequences(finder(cu, N, T, Ttot), first, step, [&](long n) {
      if (k == most) throw Enough();
      at[k++] = n;
    });
  } catch (Enough) {
    return -1;
  }
  return k;
}
// A table of N + 1 offsets in pages that are zero until the last ones: tokens belong to the last sequence.
extern "C" int last_of(int N) {
  const size_t bytes = ((size_t)N + 1) * 4;
  int32_t* cu = (int32_t*)mmap(nullptr, bytes, PROT_READ | PROT_WRITE, MAP_PRIVATE | MAP_ANONYMOUS | MAP_NORESERVE, -1, 0);
  if (cu == MAP_FAILED) return -2;
  cu[N] = 5;
  int start, end;
  const int n = finder(cu, N, 0, 5).find(3, start, end);
  munmap(cu, bytes);
  return n;
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    at = tmp_path_factory.mktemp("sequences")
    src, out = at / "sequences.cpp", at / "sequences.so"
    src.write_text(SEQUENCES)
    subprocess.run([build.hipcc(), "-x", "hip", "--offload-host-only", "-O1", "-std=c++17", "-fPIC", "-shared", "-I", build.CSRC,
                    "-I", os.path.join(build.ROOT, "include"), str(src), "-o", str(out)], check=True)
    lib = ctypes.CDLL(str(out))
    lib.met.restype = ctypes.c_long
    lib.met.argtypes = [ctypes.c_void_p] + [ctypes.c_int] * 3 + [ctypes.c_long] * 3 + [ctypes.c_void_p]
    return lib


def met(lib, cu, N, T, total, first, step, most=4096):
    at = (ctypes.c_long * most)()
    k = lib.met(None if cu is None else (ctypes.c_int32 * len(cu))(*cu), N, T, total, first, step, most, at)
    assert k >= 0, "a share that does not end"
    return list(at[:k])


def test_shares_meet_each_empty_sequence_once(lib):
    rng = random.Random(7)
    for _ in range(500):
        T, N, shares = rng.choice([0, 1, 20]), rng.randint(1, 40), rng.randint(1, 30)
        cu = sorted(rng.randint(0, T) for _ in range(N + 1))
        found = [n for s in range(shares) for n in met(lib, cu, N, 0, T, s, shares)]
        assert sorted(found) == [n for n in range(N) if cu[n] == cu[n + 1]]
    assert [n for s in range(3) for n in met(lib, None, 7, 5, 35, s, 3)] == []          # rows of five tokens
    assert sorted(n for s in range(3) for n in met(lib, None, 7, 0, 0, s, 3)) == list(range(7))


@pytest.mark.parametrize("N", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 2 ** 20])
def test_shares_of_the_most_sequences_end(lib, N):
    step = 2 ** 23 + 3                          # the last one's number plus a step leaves an int
    for first in (0, 5, step - 1):
        assert met(lib, None, N, 0, 0, first, step) == list(range(first, N, step))


@pytest.mark.parametrize("N", [5, 2 ** 30 + 9, 2 ** 31 - 2])
def test_the_last_of_many_sequences_is_found(lib, N):
    assert lib.last_of(N) == N - 1
