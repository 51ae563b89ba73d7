"""Which blocks' parts the join of a split segment takes: the blocks it passes and the one it ends in,
and never a block that does not exist or that another segment's part lies in, also when a block in
between ended early (its wait ran out). Compiled for the host from the kernels' own header."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sub_bit_quantized_gb300", "csrc")
BEGINS, GOES_ON, ENDS, NO_WORK = 0, 1, 2, 3

SOURCE = """
#include "kivi_tree_join.h"
// the kernel's walk over blocks k + 1 .. : 32 at a time; returns the state and marks the blocks read
extern "C" int walk(const int* first, int G, int k, unsigned char* read) {
  for (int base = k + 1;; base += 32) {
    unsigned on = 0, ends = 0;
    for (int i = 0; i < 32; ++i) {
      const int f = base + i < G ? first[base + i] : kvq::kSegNoWork;
      on |= (unsigned)(f == kvq::kSegGoesOn) << i;
      ends |= (unsigned)(f == kvq::kSegEnds) << i;
    }
    const kvq::JoinParts j = kvq::join_parts(on, ends);
    for (int i = 0; i < 32; ++i)
      if (j.parts >> i & 1u) {
        if (base + i >= G) return -1;  // read past the last block
        read[base + i] = 1;
      }
    if (j.state) return j.state;
  }
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    d = tmp_path_factory.mktemp("join")
    (d / "walk.cpp").write_text(SOURCE)
    so = d / "walk.so"
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(d / "walk.cpp"), "-o", str(so)], check=True)
    f = ctypes.CDLL(str(so)).walk

    def run(first, k):
        G = len(first)
        read = (ctypes.c_ubyte * G)()
        state = f((ctypes.c_int * G)(*first), G, k, read)
        return state, [i for i in range(G) if read[i]]
    return run


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 64, 65, 300])
@pytest.mark.parametrize("k", [0, 5])
def test_whole_segments(walk, n, k):
    # the segment that block k opens passes n - 1 blocks and ends in the next; other segments follow
    first = [BEGINS] * (k + 1) + [GOES_ON] * (n - 1) + [ENDS] + [BEGINS, ENDS, GOES_ON] + [NO_WORK] * 3
    assert walk(first, k) == (1, list(range(k + 1, k + n + 1)))
    assert walk(first[:k + n + 1], k) == (1, list(range(k + 1, k + n + 1)))  # it ends in the last block


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 64, 70])
@pytest.mark.parametrize("left", [BEGINS, NO_WORK])
def test_cut_off_segments(walk, n, left):
    # block k + n ended early; behind it other segments end and go on
    for tail in ([ENDS, GOES_ON, ENDS], [GOES_ON] * 40 + [ENDS], []):
        first = [BEGINS] + [GOES_ON] * (n - 1) + [left] + tail
        assert walk(first, 0) == (2, list(range(1, n)))


@pytest.mark.parametrize("n", [0, 1, 31, 32, 64, 303])
def test_segments_without_an_end(walk, n):
    # the block it should end in is missing from the records: nothing past the last block is read
    assert walk([BEGINS] + [GOES_ON] * n, 0) == (2, list(range(1, n + 1)))
